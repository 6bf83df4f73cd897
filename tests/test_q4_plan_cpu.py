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


def decode(driver, cases):
    """[(cluster, splits)] of cases (D, groups, keys in falling order)."""
    got = driver([f"decode {d} {g} {' '.join(map(str, HELD))} {len(keys)} {' '.join(map(str, keys))}" for d, g, keys in cases])
    return [(line[0], line[1:]) for line in got]


def check_plan(groups, keys, cluster, splits):
    chunks = [(k + 31) // 32 for k in keys]
    ctas = groups * sum(splits)
    assert 1 <= cluster <= 13 and all(1 <= s <= cluster and cluster % s == 0 for s in splits)
    # No CTA without a chunk of its own; equal splits are chosen by the longest
    # sequence, and shorter ones beside it may leave CTAs without keys.
    shared = zip(splits, chunks) if len(set(splits)) > 1 else [(splits[0], chunks[0])]
    assert all(s == 1 or s <= c for s, c in shared)
    if len(set(splits)) == 1 and cluster > 1:
        assert ctas <= cluster * HELD[cluster - 1]                          # all clusters at once
    assert splits == sorted(splits, reverse=True)                           # no group straddles a cluster


def test_splits_of_equal_sequences(driver):
    cases = [(d, g, [k] * n) for d in (64, 128) for g in (1, 2, 8, 16, 5000) for n in (1, 3, 24, 64)
             for k in (0, 1, 31, 32, 33, 256, 512, 2048, 16384, 1 << 24)]
    for (d, g, keys), (cluster, splits) in zip(cases, decode(driver, cases)):
        check_plan(g, keys, cluster, splits)
        assert set(splits) == {cluster}
    # the two sides of the rule, and a launch that is larger than the device
    short, long, many = decode(driver, [(128, 8, [2048] * 4), (128, 8, [16384] * 4), (128, 5000, [16384])])
    assert short[0] == 4 and long[0] == 8 and many[0] == 1


def test_splits_of_mixed_sequences(driver):
    rng = random.Random(5)
    cases = []
    for _ in range(400):
        n = rng.randint(1, 64)
        top = rng.choice([300, 3000, 16384, 100000])
        cases.append((rng.choice([64, 128]), rng.choice([1, 2, 4, 8, 16]), sorted((int(top ** rng.random()) for _ in range(n)), reverse=True)))
    mixed = 0
    for (d, g, keys), (cluster, splits) in zip(cases, decode(driver, cases)):
        check_plan(g, keys, cluster, splits)
        mixed += len(set(splits)) > 1
    assert mixed > 40


def test_key_parts_cover_every_tile_once(driver):
    rng = random.Random(7)
    cases = []
    for _ in range(600):
        seqs = [(int(80000 ** rng.random()), int(600 ** rng.random()) + 17) for _ in range(rng.randint(1, 5))]
        window = rng.choice([0, 0, 1, 200, 1000, 5000, 20000])
        cases.append((window, rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 8]), seqs))
    got = driver([f"parts {w} {d} {g} {h} 152 {len(s)} {' '.join(f'{a} {b}' for a, b in s)}" for w, d, g, h, s in cases])
    cut = 0
    for (window, d, g, hkv, seqs), (yes, hpi, *flat) in zip(cases, got):
        if not yes:
            continue
        cut += 1
        parts = list(zip(flat[0::3], flat[1::3], flat[2::3]))
        assert len(parts) <= 8 and hpi in (1, 2) and g % hpi == 0
        blocks = [-(-n // 128) for _, n in seqs]
        assert sum(blocks[r] for r, _, _ in parts) * hkv * (g // hpi) <= 152       # one item an SM
        assert sum(seqs[r][1] for r, _, _ in parts) * hkv * g <= 256 * 152         # what the cache has room for
        assert sorted(r for r, _, _ in parts) == [r for r, _, _ in parts] and {r for r, _, _ in parts} == set(range(len(seqs)))
        for i, (start, n) in enumerate(seqs):
            mine = [(lo, hi) for r, lo, hi in parts if r == i]
            for b in range(blocks[i]):
                pos = start + 128 * b
                first = max(0, pos + 1 - window) // 128 if window else 0
                end = (start + min(n, 128 * b + 128) - 1) // 128 + 1
                seen = [t for lo, hi in mine for t in range(max(lo, first), min(hi, end))]
                assert seen == list(range(first, end))
                assert all(max(lo, first) < min(hi, end) for lo, hi in mine)           # none without a tile
    assert cut > 150


def test_key_parts_where_they_pay(driver):
    one = [f"parts 0 128 4 8 152 1 {start} {n}" for start, n in ((16384, 128), (2048, 128), (1000, 128), (2048, 512), (0, 128))]
    assert [line[0] for line in driver(one)] == [1, 1, 0, 0, 0]
    assert driver(["parts 0 128 8 1 152 1 16384 128", "parts 0 128 4 8 152 1 16384 128"]) == [
        [1, 1] + [x for k in range(8) for x in (0, 129 * k // 8, 129 * (k + 1) // 8 if k < 7 else 1 << 30)],
        [1, 2] + [x for k in range(8) for x in (0, 129 * k // 8, 129 * (k + 1) // 8 if k < 7 else 1 << 30)]]


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
