"""The launch record (csrc/launch_order.h) keeps streams apart that share a handle,
on the CPU through a small driver built with g++: the default streams of two
devices, and the per-thread default streams of two threads.  What is recorded for
one must leave the guard of the other's launches alone.  Nor do launches that go
into a graph end what the stream that captures them still runs."""
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
    exe = str(tmp_path_factory.mktemp("streams") / "launch_streams_driver")
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "native", "launch_streams_driver.cpp"),
                    "-o", exe, "-lpthread"], check=True)

    def run(*lines):
        out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True, timeout=60)
        return [int(x) for x in out.stdout.split()]
    return run


@pytest.mark.parametrize("handle", [0, 1, 77])
def test_a_barrier_or_a_synchronisation_of_another_device(driver, handle):
    here, there = f"{handle} 0 0", f"{handle} 1 0"
    assert driver(f"admit {here} 10", f"barrier {there}", f"settled {here}", f"admit {here} 10") == [0, 0, 1]
    assert driver(f"admit {here} 10", "clear 1", f"settled {here}", f"admit {here} 10") == [0, 0, 1]
    assert driver(f"admit {here} 10", f"barrier {here}", f"settled {here}", f"admit {here} 10") == [0, 1, 0]
    assert driver(f"admit {here} 10", "clear 0", f"settled {here}", f"admit {here} 10") == [0, 1, 0]


@pytest.mark.parametrize("handle", [0, 77])
def test_blocks_of_another_device_are_not_resident_here(driver, handle):
    # 304 blocks on the other device do not end this one's walk
    here, there = f"{handle} 0 0", f"{handle} 1 0"
    assert driver(f"admit {here} 10", f"admit {there} 304", f"settled {here}", f"admit {here} 10") == [0, 0, 0, 1]


def test_the_two_handles_of_the_legacy_stream_are_one(driver):
    assert driver("admit 0 0 0 10", "settled 1 0 0", "admit 1 0 0 10") == [0, 0, 1]
    assert driver("admit 0 0 0 10", "barrier 1 0 0", "settled 0 0 0") == [0, 1]


def test_each_thread_has_its_own_per_thread_stream(driver):
    assert driver("admit 2 0 0 10", "barrier 2 0 1", "admit 2 0 0 10") == [0, 1]
    assert driver("admit 2 0 0 10", "admit 2 0 1 304", "admit 2 0 0 10") == [0, 0, 1]
    # any other stream is the same in every thread
    assert driver("admit 77 0 0 10", "settled 77 0 1", "barrier 77 0 1", "settled 77 0 0") == [0, 0, 1]


def test_captured_launches_do_not_hide_what_the_stream_still_runs(driver):
    # 304 captured blocks, and a captured kernel that never signals early, between
    # two steps of one layer that run: the second's guard still counts the first
    # (and the captured step's row)
    run, captured = "77 0 0", "77 0 0 {} 5"
    assert driver(f"admit {run} 10", f"admit {captured.format(304)}", f"settled {run}", f"admit {run} 10") == [0, 0, 0, 2]
    assert driver(f"admit {run} 10", f"barrier {captured.format(0)}", f"settled {run}", f"admit {run} 10") == [0, 0, 1]


def test_captured_launches_are_ordered_among_themselves(driver):
    first, second = "77 0 0 {} 5", "77 0 0 {} 6"
    assert driver("admit 77 0 0 10", f"settled {first.format(0)}", *[f"admit {first.format(10)}"] * 3,
                  f"settled {first.format(0)}", f"barrier {first.format(0)}", f"admit {first.format(10)}") == [0, 1, 0, 1, 2, 0, 0]
    # the next capture on the stream starts anew
    assert driver(f"admit {first.format(10)}", f"settled {second.format(0)}", f"barrier {second.format(0)}",
                  f"admit {second.format(10)}", f"admit {second.format(10)}") == [0, 1, 0, 1]
    # a synchronisation is of what runs
    assert driver(f"admit {first.format(10)}", "admit 77 0 0 10", "clear 0", f"settled {first.format(0)}", "settled 77 0 0") == [0, 1, 0, 1]
