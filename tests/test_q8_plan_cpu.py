"""Which rows the 8-bit cache keeps in bf16 (csrc/q8_tail.h) and how its steps are
cut (csrc/q8_plan.h), on the CPU through a small driver built with g++."""
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gqa_attention_preallocated_qa_gb300", "csrc")
BLOCK = 64


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("plan") / "q8_plan_driver")
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "native", "q8_plan_driver.cpp"),
                    "-o", exe], check=True)
    return exe


@pytest.fixture(scope="module")
def ask(exe):
    p = subprocess.Popen([exe], stdin=subprocess.PIPE, stdout=subprocess.PIPE, text=True)

    def one(*words):
        p.stdin.write(" ".join(map(str, words)) + "\n")
        p.stdin.flush()
        return [int(x) for x in p.stdout.readline().split()]
    yield one
    p.stdin.close()
    p.wait(10)


class Model:
    """One (sequence, kv head): what every row is (a version that counts the writes, or
    ("codes", version) where it came back from the codes), written as the kernels write."""

    def __init__(self, ask):
        self.ask = ask
        self.state = [-1, -1, -1, -1, -1, -1]
        self.buf = [[None] * BLOCK, [None] * BLOCK]
        self.codes = {}
        self.last = {}     # position -> version last written
        self.n = 0

    def row(self, blk, r, raw):
        i = self.ask("of", *self.state, blk, r, int(raw))[0]
        return self.buf[i][r] if i >= 0 else self.codes.get((blk, r))

    def write(self, start, end, step):
        self.n += 1
        first, last = start // BLOCK, (end - 1) // BLOCK
        src, from_rows, dst, *nxt = self.ask("tail", *self.state, start, end, int(step))
        # where the earlier rows of the first block come from
        old = {}
        for r in range(start % BLOCK):
            if src >= 0 and r < from_rows:
                assert self.state[3 * src] == first
                old[r] = self.buf[src][r]
            else:
                held = self.codes.get((first, r))
                old[r] = held if held is None or isinstance(held, tuple) else ("codes", held)
        for p in range(start, end):
            self.last[p] = self.n
        for b in range(first, last + 1):
            if end >= (b + 1) * BLOCK:
                for r in range(BLOCK):
                    p = b * BLOCK + r
                    self.codes[b, r] = self.n if p >= start else old[r]
        if dst >= 0:
            assert nxt[3 * dst] == last
            if src >= 0 and last > first and from_rows > 0:
                assert dst != src  # it is read while the other is written
            for r in range(end - last * BLOCK):
                p = last * BLOCK + r
                if p >= start:
                    self.buf[dst][r] = self.n
                elif r >= from_rows or dst != src:
                    self.buf[dst][r] = old[r]
        self.state = nxt

    def check(self, end):
        """Every buffered row and every row below `end` is what was last written there."""
        for i in range(2):
            b, rows, sealed = self.state[3 * i:3 * i + 3]
            if b >= 0:
                assert 1 <= rows <= BLOCK
                for r in range(rows):
                    got = self.buf[i][r]
                    version = got[1] if isinstance(got, tuple) else got
                    assert version == self.last.get(b * BLOCK + r), (b, r)
        assert self.state[0] < 0 or self.state[0] != self.state[3]
        for p in range(max(0, end - 200), end):
            got = self.row(p // BLOCK, p % BLOCK, False)
            got = got[1] if isinstance(got, tuple) else got
            assert got == self.last[p], p


@pytest.mark.parametrize("seed", range(12))
def test_no_write_leaves_a_row_behind(ask, seed):
    rng = random.Random(seed)
    m, end = Model(ask), 0
    for _ in range(250):
        kind = rng.random()
        if kind < 0.5:                      # a step, mostly where the sequence ends
            start = end
            if rng.random() < 0.25:
                start = max(0, end - rng.choice([1, 2, 5, 60, 64, 70, 130, 200]))
            m.write(start, start + 1, True)
            end = start + 1
        else:                               # rows
            start = end if rng.random() < 0.6 else rng.randint(0, end)
            n = rng.choice([1, 2, 10, 63, 64, 65, 128, 150])
            m.write(start, start + n, False)
            end = start + n
        m.check(end)


def test_rows_survive_a_step_back_into_the_block_before(ask):
    m = Model(ask)
    for p in range(70):
        m.write(p, p + 1, True)
    m.write(62, 63, True)   # a row of the block before the current one
    assert not any(isinstance(x, tuple) for i in range(2) for x in m.buf[i][:63] if m.state[3 * i] == 0)
    m.check(63)
    # two blocks back the rows come from the codes
    for p in range(63, 200):
        m.write(p, p + 1, True)
    m.write(10, 11, True)
    i = m.ask("of", *m.state, 0, 5, 1)[0]
    assert i >= 0 and isinstance(m.buf[i][5], tuple)


def test_the_same_rows_written_again_leave_the_same_state(ask):
    """A call that is repeated finds the rows before it as they were."""
    for start, end in ((17, 300), (64, 130), (130, 131), (63, 64), (5, 60), (1, 65), (130, 2178)):
        m = Model(ask)
        if start:
            m.write(0, start, False)
        before = [m.row(start // BLOCK, r, True) for r in range(start % BLOCK)]
        for _ in range(3):
            m.write(start, end, end - start == 1)
            m.check(end)
            assert [m.row(start // BLOCK, r, True) for r in range(start % BLOCK)] == before


def test_splits_of_a_step(ask):
    rng = random.Random(3)
    for _ in range(400):
        n = rng.randint(1, 64)
        hkv = rng.choice([1, 2, 3, 4, 8, 40])
        work = sorted((rng.randint(0, rng.choice([1, 8, 100, 3000])) for _ in range(n)), reverse=True)
        top, *splits = ask("step", 152, hkv, 16, n, *work)
        assert top == max(splits) <= 16 and all(s & (s - 1) == 0 and top % s == 0 for s in splits)
        assert splits == sorted(splits, reverse=True)
        assert all(s == 1 or 4 * (s // 2) < w for s, w in zip(splits, work))  # no CTA without work
        assert hkv * sum(splits) <= 304 or top == 1
    # one short sequence, the four-prompt step, long caches
    assert ask("step", 152, 8, 16, 1, 8)[0] == 2
    assert ask("step", 152, 8, 16, 4, 32, 32, 32, 32)[0] == 4
    assert ask("step", 152, 8, 16, 4, 256, 256, 256, 256)[0] == 8
    assert ask("step", 152, 8, 16, 1, 256)[0] == 16
    assert ask("step", 152, 1, 16, 1, 0) == [1, 1]


def test_work_of_a_step(ask):
    assert ask("work", 128, 100, 0) == [100]
    assert ask("work", 64, 101, 0) == [51]
    assert ask("work", 128, 100, 100) == [100]
    assert ask("work", 128, 1024, 32) == [64]
    # never less for a longer sequence: the plan takes them in falling order
    for n in (1, 16, 64):
        got = [ask("work", 128, full, n)[0] for full in range(0, 400)]
        assert got == sorted(got)
