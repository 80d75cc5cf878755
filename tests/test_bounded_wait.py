"""The kernels' bounded wait, compiled for the host: a wait that nothing ends gives up after a fixed number
of tries, and once one has, every later one gives up after a single try."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "vision_selective_state_b200", "csrc")

SOURCE = r"""
#include <cstdio>
#include "vscan_tc.cuh"

int main()
{
    using vscan::TC_WAIT_TRIES;
    volatile int dead = 0;
    long long tries = 0;
    auto never = [&] { ++tries; return false; };
    auto after = [&](long long n) { return [&tries, n] { return ++tries > n; }; };
    // waits that end in time, at once and late: as many tries as it takes, and no mark
    for (long long n : {0LL, 1LL, 255LL, 256LL, 257LL, 100000LL, (long long)TC_WAIT_TRIES - 1}) {
        tries = 0;
        vscan::tc_bounded_wait(after(n), &dead);
        printf("%lld %d\n", tries - n - 1, dead);
    }
    // one that does not
    tries = 0;
    vscan::tc_bounded_wait(never, &dead);
    printf("%lld %d\n", tries - TC_WAIT_TRIES, dead);
    // the later ones of the same block
    for (int i = 0; i < 3; ++i) {
        tries = 0;
        vscan::tc_bounded_wait(never, &dead);
        printf("%lld %d\n", tries - 1, dead);
    }
    // one that another thread's giving up ends while it waits
    dead = 0;
    tries = 0;
    vscan::tc_bounded_wait([&] { if (++tries == 1000) dead = 1; return false; }, &dead);
    printf("%d %d\n", tries > 1000 + 256, dead);
    return 0;
}
"""


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    at = tmp_path_factory.mktemp("wait")
    (at / "wait.cu").write_text(SOURCE)
    subprocess.run(["nvcc", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-cudart", "static", "-I", CSRC,
                    "-o", str(at / "wait"), str(at / "wait.cu")], check=True, capture_output=True)
    out = subprocess.run([str(at / "wait")], check=True, capture_output=True, text=True, timeout=60).stdout
    return [tuple(int(x) for x in line.split()) for line in out.splitlines()]


def test_waits_that_end_take_their_tries_and_leave_no_mark(lines):
    assert lines[:7] == [(0, 0)] * 7


def test_a_wait_that_nothing_ends_gives_up_and_marks_it(lines):
    assert lines[7] == (0, 1)


def test_later_waits_give_up_after_one_try(lines):
    assert lines[8:11] == [(0, 1)] * 3


def test_a_wait_ends_soon_after_another_gave_up(lines):
    assert lines[11] == (0, 1)
