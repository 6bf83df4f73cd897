"""How the 4-bit cache's launches are cut (csrc/q4_plan.h), on the CPU through a
small driver built with g++: a decode step's splits and a prefill's runs."""
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gqa_attention_preallocated_qa_gb300", "csrc")
# Clusters of S = 1..13 CTAs that one GB300 holds at once, two CTAs per SM.
HELD = [304, 152, 97, 74, 58, 46, 38, 36, 30, 28, 23, 23, 19]


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("plan") / "q4_plan_driver")
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "native", "q4_plan_driver.cpp"),
                    "-o", exe], check=True)

    def run(lines):
        out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True)
        return [[int(x) for x in line.split()] for line in out.stdout.splitlines()]
    return run


def test_splits_fit_and_have_work(driver):
    cases = [(d, g, k) for d in (64, 128) for g in (1, 8, 16, 32, 48, 96, 128, 192, 300, 5000)
             for k in (0, 1, 31, 32, 33, 256, 512, 2048, 16384, 1 << 24)]
    got = driver([f"splits {d} {g} {k} " + " ".join(map(str, HELD)) for d, g, k in cases])
    for (d, g, k), (s,) in zip(cases, got):
        assert 1 <= s <= 13
        assert s == 1 or (HELD[s - 1] >= g and s <= (k + 31) // 32), (d, g, k, s)
    one = dict(zip(cases, (s for s, in got)))
    assert one[(128, 32, 2048)] == 4 and one[(128, 32, 16384)] == 8  # the two sides of the rule
    assert one[(128, 5000, 16384)] == 1


def test_runs_cover_every_row_once_and_never_cost_more(driver):
    rng = random.Random(3)
    cases = []
    for _ in range(300):
        n = rng.randint(1, 8)
        cases.append((rng.choice([0, 0, 700]), 8, [(rng.choice([0, rng.randint(1, 6000)]), rng.randint(1, 2000)) for _ in range(n)]))
    lines = [f"runs {w} 128 4 {hkv} 152 {len(seqs)} " + " ".join(f"{s} {n}" for s, n in seqs) for w, hkv, seqs in cases]
    cut = 0
    for (w, hkv, seqs), got in zip(cases, driver(lines)):
        before, after, flat = got[0], got[1], got[2:]
        runs = [flat[i:i + 3] for i in range(0, len(flat), 3)]
        assert len(seqs) <= len(runs) <= 8
        rows = {(q, r) for q, first, n in runs for r in range(first, first + n)}
        assert sum(n for _, _, n in runs) == len(rows) == sum(n for _, n in seqs)
        assert all(first % 128 == 0 and n > 0 for _, first, n in runs)
        # a run that is not its sequence's last is whole blocks
        assert all(n % 128 == 0 or first + n == seqs[q][1] for q, first, n in runs)
        starts = {s for s, _ in seqs}
        assert after <= before
        if len(runs) > len(seqs):
            assert len(starts) > 1 and after < before
            cut += 1
    assert cut > 30


def test_runs_of_equal_starts_are_left_whole(driver):
    (got,) = driver(["runs 0 128 4 8 152 4 0 2048 0 2048 0 2048 0 2048"])
    assert got[2:] == [0, 0, 2048, 1, 0, 2048, 2, 0, 2048, 3, 0, 2048]
