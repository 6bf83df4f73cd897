"""What a synchronisation of the device says about the launches of threads that have ended
(csrc/launch_order.h): what was enqueued before it has finished, whoever launched it, and
its record goes.  On the CPU through a small driver built with g++."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gqa_attention_preallocated_qa_gb300", "csrc")
KEPT = 1 << 14  # launches that a record holds


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("ended") / "launch_ended_driver")
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "native", "launch_ended_driver.cpp"),
                    "-o", exe, "-lpthread"], check=True)

    def run(*lines):
        out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True, timeout=60)
        return [int(x) for x in out.stdout.split()]
    return run


@pytest.mark.parametrize("handle", [2, 77])
def test_threads_that_have_ended_leave_nothing(driver, handle):
    """On their per-thread streams (2), and on one that they shared."""
    assert driver(f"threads 50 {handle}", "settled", "mark", "clear", "settled") == [0, 50]


def test_what_came_after_the_mark_stays(driver):
    assert driver("threads 3 2", "mark", "threads 4 2", "clear", "settled") == [3]
    assert driver("threads 3 77", "mark", "threads 1 77", "clear", "settled", "stream 77") == [0, 0]
    # this thread's own launches have finished with its synchronisation, in any case
    assert driver("mark", "launch 77", "clear", "stream 77") == [1]


def test_a_call_that_is_under_way_stays(driver):
    """Its launch is recorded and may not have been made."""
    assert driver("threads 2 2", "calls 3 2", "threads 1 2", "mark", "clear", "settled", "go",
                  "mark", "clear", "settled") == [2, 6]


def test_a_full_record_of_ended_threads_ends_too(driver):
    """More launches than it holds, by two threads: those that fell out have finished as well."""
    fill = ["launch 77"] * (KEPT + 5)
    assert driver("threads 1 77", *fill, "threads 1 77", "mark", "clear", "stream 77") == [1]
    assert driver("threads 1 77", *fill, "mark", "threads 1 77", "clear", "stream 77") == [0]
