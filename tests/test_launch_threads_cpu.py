"""What a thread's synchronisation of the device says about another thread's launches
(csrc/launch_order.h): nothing.  On the CPU through a small driver built with g++."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gqa_attention_preallocated_qa_gb300", "csrc")


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("threads") / "launch_threads_driver")
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "native", "launch_threads_driver.cpp"),
                    "-o", exe, "-lpthread"], check=True)

    def run(*lines):
        out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True, timeout=60)
        return [int(x) for x in out.stdout.split()]
    return run


def test_another_threads_launches_stay(driver):
    """Thread 1 frees a cache, or asks for an error, while thread 0's step still runs."""
    assert driver("admit 0 1 3 1", "clear 1", "settled 1 3", "admit 0 1 3 1") == [0, 0, 1]
    assert driver("admit 0 1 3 1", "clear 0", "settled 1 3", "admit 0 1 3 1") == [0, 1, 0]
    assert driver("admit 0 1 3 1", "admit 1 2 4 1", "clear 1", "settled 1 3", "settled 2 4") == [0, 0, 0, 1]


def test_a_stream_of_two_threads(driver):
    """The one's launches have finished, the other's may run."""
    assert driver("admit 0 1 3 1", "admit 1 1 4 1", "clear 1", "settled 1 3", "settled 1 4") == [0, 0, 0, 1]
    assert driver("admit 0 1 3 1", "admit 1 1 4 1", "clear 0", "settled 1 3", "settled 1 4") == [0, 0, 1, 0]
    # both, one after the other: nothing is left
    assert driver("admit 0 1 3 1", "admit 1 1 4 1", "clear 0", "clear 1", "settled 1 3", "settled 1 4") == [0, 0, 1, 1]
    # a launch that waited before it signalled bounds the walk only while it is there
    assert driver("admit 0 1 3 1", "admit 1 1 4 0", "settled 1 3", "clear 1", "settled 1 3") == [0, 0, 1, 0]


def test_more_launches_than_are_kept(driver):
    """What fell out of a shared record is not known to have finished."""
    many = ["admit 0 1 5 1"] * ((1 << 14) + 1)
    got = driver("admit 1 1 3 1", *many, "clear 0", "settled 1 3")
    assert got[-1] == 0
