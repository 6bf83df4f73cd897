"""The launch record (csrc/launch_order.h) of a capture whose streams wait for each
other's events: the graph's edge from the other stream's launch is programmatic, so a
launch that follows it may start beside it and everything that it ran beside.  On the
CPU through a small driver built with g++."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gqa_attention_preallocated_qa_gb300", "csrc")
ALL = 1 << 30


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("forks") / "launch_forks_driver")
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "native", "launch_forks_driver.cpp"),
                    "-o", exe, "-lpthread"], check=True)

    def run(*lines):
        out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True, timeout=60)
        return [int(x) for x in out.stdout.split()]
    return run


# stream 1 captures; its first launch writes layer 0 and becomes node 11
FIRST = "admit 1 5 0 1 - 11"


def test_a_stream_that_follows_anothers_launch(driver):
    # stream 2 has waited for an event behind node 11: nothing is settled there
    assert driver(FIRST, "settled 2 5 0 11", "settled 2 5 1 11", "inflight 2 5 0 11", "admit 2 5 0 1 11 12") == [0, 0, 0, 2, ALL]
    # what follows on it may run beside node 11 as well, unless a launch lies between that waited first
    assert driver(FIRST, "admit 2 5 1 1 11 12", "settled 2 5 0 12", "admit 2 5 0 1 12 13") == [0, ALL, 0, ALL]
    assert driver(FIRST, "admit 2 5 1 0 11 12", "settled 2 5 0 12", "admit 2 5 0 1 12 13") == [0, ALL, 1, 0]


def test_a_stream_that_joins_another(driver):
    fork = (FIRST, "admit 2 5 1 0 11 12")
    # stream 1 goes on by itself, then waits for node 12
    assert driver(*fork, "admit 1 5 2 1 11 13", "settled 1 5 0 13", "settled 1 5 1 13", "settled 1 5 1 13,12",
                  "settled 1 5 2 12", "admit 1 5 3 1 12,13 14", "settled 1 5 1 14") == [0, ALL, 0, 0, 1, 0, 0, ALL, 0]
    # a launch that waited first ends it
    assert driver(*fork, "admit 1 5 3 0 11,12 14", "settled 1 5 1 14") == [0, ALL, ALL, 1]


def test_other_codes_nodes_are_no_launches_of_ours(driver):
    # 90: a kernel of other code, which follows node 11, or nothing
    assert driver(FIRST, "settled 2 5 0 90", "settled 1 5 0 90", "settled 1 5 1 90") == [0, 1, 0, 1]
    assert driver(FIRST, "admit 1 5 0 1 11,90 12", "admit 1 5 0 1 12 13") == [0, 1, 2]


def test_a_barrier_forgets_its_streams_launches_alone(driver):
    # node 11 is still there to be followed
    assert driver(FIRST, "barrier 1 5 11", "settled 1 5 0 91", "settled 2 5 0 11", "settled 2 5 0 91") == [0, 1, 0, 1]
    assert driver(FIRST, "admit 2 5 1 1 11 12", "barrier 2 5 12", "settled 2 5 0 92") == [0, ALL, 1]


def test_captures_are_kept_apart(driver):
    # the same node number in another capture, and in a stream that runs
    assert driver(FIRST, "settled 2 6 0 11", "settled 1 6 0 11", "settled 2 0 0 -") == [0, 1, 1, 1]
