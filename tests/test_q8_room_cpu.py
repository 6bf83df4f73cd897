"""Steps of the 8-bit cache whose thread blocks have an SM to themselves, for their shared
memory (csrc/q8_plan.h): the plan does not count on two.  On the CPU through a small driver
built with g++."""
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gqa_attention_preallocated_qa_gb300", "csrc")
KB = 1024


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("room") / "q8_room_driver")
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "native", "q8_room_driver.cpp"),
                    "-o", exe], check=True)

    def one(*words):
        out = subprocess.run([exe], input=" ".join(map(str, words)) + "\n", capture_output=True, text=True, check=True)
        return [int(x) for x in out.stdout.split()]
    return one


def test_ctas_that_fit_an_sm(ask):
    for cta, fit in ((77 * KB, 2), (113 * KB, 2), (113 * KB + 1, 1), (170 * KB, 1)):
        assert ask("room", 228 * KB, KB, cta) == [fit]


def test_one_cta_an_sm_is_one_wave(ask):
    rng = random.Random(5)
    for _ in range(60):
        n, hkv = rng.randint(1, 20), rng.choice([1, 2, 4, 8, 16])
        work = sorted((rng.randint(1, 3000) for _ in range(n)), reverse=True)
        top, *splits = ask("step", 152, 1, hkv, 16, n, *work)
        assert top == max(splits) and splits == sorted(splits, reverse=True)
        assert hkv * sum(splits) <= 152 or top == 1
        two, *more = ask("step", 152, 2, hkv, 16, n, *work)
        assert two >= top and all(a >= b for a, b in zip(more, splits))
    # what two an SM would share out further
    assert ask("step", 152, 2, 8, 16, 4, 256, 256, 256, 256) == [8, 8, 8, 8, 8]
    assert ask("step", 152, 1, 8, 16, 4, 256, 256, 256, 256) == [4, 4, 4, 4, 4]
