"""When a tile of the recurrence gives up waiting for another one (CPU only): the rule of
csrc/scan_wait.h, compiled for the host.  Results of a wait that was given up are NaN, so a
wave that was merely not running must not give up, and one whose word never comes must."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunk_weight_rnn_amd", "csrc")


@pytest.fixture(scope="module")
def gives_up(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("wait")
    src = d / "w.cpp"
    src.write_text('#include <cstdio>\n#include <cstdlib>\n#include "scan_wait.h"\nint main(int n, char** v) {\n'
                   '  for (int i = 1; i + 1 < n; i += 2)\n'
                   '    std::printf("%d ", (int)e2ttt::gives_up((unsigned)std::strtoul(v[i], 0, 10), std::strtoull(v[i + 1], 0, 10)));\n}\n')
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, str(src), "-o", str(d / "w")], check=True)
    return lambda *pairs: [int(x) for x in subprocess.run([str(d / "w")] + [str(x) for p in pairs for x in p], capture_output=True,
                                                          text=True, check=True).stdout.split()]


SECOND = 100_000_000  # ticks


def test_a_wave_that_was_set_aside_goes_on(gives_up):
    """A few looks before and after, and seconds or hours between: the word may be about to come."""
    assert gives_up((64, 3 * SECOND), (128, 3600 * SECOND), (100_000, 10 * SECOND)) == [0, 0, 0]


def test_quick_looks_alone_do_not_end_a_wait(gives_up):
    assert gives_up((1 << 30, SECOND // 10)) == [0]


def test_every_wait_ends(gives_up):
    """Looks and the clock both go on as long as the wave runs: after 2^22 looks, some seconds, it has given up."""
    assert gives_up((1 << 22, 3 * SECOND), ((1 << 32) - 64, 3 * SECOND)) == [1, 1]


def test_the_kernel_waits_by_this_rule():
    text = open(os.path.join(CSRC, "scan.hip")).read()
    assert '#include "scan_wait.h"' in text and "gives_up(tries, now - since)" in text
    assert "kSpinTicks" not in text  # no other limit beside it
