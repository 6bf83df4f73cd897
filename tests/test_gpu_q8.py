"""The 8-bit cache on the GPU against its definition (q8_ref.py).

Tolerances, from the roundings alone.  A decode step multiplies the codes themselves,
which fp16 holds, with queries scaled by a power of two, which fp16 holds down to 2^-22
of a row's largest value.  The weights P are rounded to fp16, relative to a reference
that is at most 2^8 below the largest: 2^-11 of a weight, or 2^-25 of the largest weight where
that is more.  Scores are fp32 sums in which every code carries 128 that is taken
away again: with terms below 2^-24 (2^8 + 2^7) of the largest query, 8 sums of 2^-23 each,
that is below 2^-13 of a weight for the queries and keys here (sum |q| below 2^7, s below 2^-4,
log2(e) / sqrt(D) below 0.19).  Numerator and denominator use the same weights, so an
output moves by at most 2 (2^-11 + 2^-13) sum p |v| + 2^-24 sum |v| / l, and then one
rounding to bf16, 2^-8 |out|.  The bf16 rows' weights are sums of two bf16 numbers (2^-16),
inside that bound.  The prefill kernel rounds P to bf16: 2^-8 in the place of 2^-11.
"""
import numpy as np
import pytest
import torch

import q8_ref
from gpu_util import f64

pytestmark = pytest.mark.gpu

THETA, EPS = 1e6, 1e-6
BLOCK = q8_ref.BLOCK


@pytest.fixture(scope="module")
def qa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gqa_attention_preallocated_qa_gb300 import _build
    _build.build()
    from gqa_attention_preallocated_qa_gb300 import binding
    return binding


def rows(seed, *shape, gain=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * gain).bfloat16()


class Cache:
    """An 8-bit cache of one layer beside what it should hold."""

    def __init__(self, qa, batch, hq, hkv, d, cap, layers=1, seed=1):
        self.qa, self.hq, self.hkv, self.d, self.cap, self.batch = qa, hq, hkv, d, cap, batch
        self.h = qa.qa_q8_cache_alloc(layers, batch, hq, hkv, d, cap, THETA, EPS)
        self.ref = q8_ref.Rows(batch, hkv, d, cap)
        self.wq, self.wk = 1 + 0.1 * rows(seed, d), 1 + 0.1 * rows(seed + 1, d)

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.qa.qa_q8_cache_free(self.h)

    def append(self, start, ntok, k, v, layer=0):
        self.qa.qa_q8_append(self.h, layer, start, ntok, k, v)
        self.ref.write(start, ntok, f64(k), f64(v))

    def fill(self, lens, seed, gain=1.0):
        k, v = rows(seed, sum(lens), self.hkv, self.d, gain=gain), rows(seed + 1, sum(lens), self.hkv, self.d)
        self.append([0] * len(lens), lens, k, v)

    def check_read(self, lens, start=None, ntok=None, layer=0):
        start = start or [0] * len(lens)
        ntok = ntok or [n - s for n, s in zip(lens, start)]
        k = torch.full((sum(ntok), self.hkv, self.d), 7.0, device="cuda", dtype=torch.bfloat16)
        v = k.clone()
        self.qa.qa_q8_read(self.h, layer, start, ntok, k, v)
        at = 0
        for b, (s, n) in enumerate(zip(start, ntok)):
            for i, x in enumerate((k, v)):
                np.testing.assert_array_equal(f64(x[at:at + n]), self.ref.read(i, b, s, n, lens[b]), err_msg=f"sequence {b}, {'kv'[i]}")
            at += n

    def tokens(self, n, seed):
        return rows(seed, n, self.hq, self.d), rows(seed + 1, n, self.hkv, self.d), rows(seed + 2, n, self.hkv, self.d)

    def want(self, b, pos, q, blocks=None):
        """Attention of q [1, Hq, D] (float64) at position pos, whose row the reference has."""
        full = pos // BLOCK
        outs, mags, flats = [], [], []
        g = self.hq // self.hkv
        k, v = (self.ref.held(i, b, pos, blocks) for i in (0, 1))
        for h in range(self.hkv):
            kk, vv = (torch.from_numpy(np.concatenate((x[h], self.ref.came[i, b, h, pos:pos + 1]))).cuda()[None]
                      for i, x in enumerate((k, v)))
            o, m, f = q8_ref.attend(q[:, h * g:(h + 1) * g], kk, vv, kk.shape[1] - 1)
            outs.append(o)
            mags.append(m)
            flats.append(f)
        assert full == pos // BLOCK
        return torch.cat(outs, 1), torch.cat(mags, 1), torch.cat(flats, 1)


def close(got, want, mag, flat, p_bits=11, what=""):
    got = got.double()
    tol = 2.0 ** -8 * want.abs() + 2 * (2.0 ** -p_bits + 2.0 ** -13) * mag + 2.0 ** -24 * flat + 1e-6
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {float(((got - want).abs() / tol).max()):.3f} of the tolerance"


# ------------------------------------------------------------------ rows
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv", [1, 3])
def test_append_and_read_are_the_definition(qa, d, hkv):
    lens = [64, 1, 63, 65, 200, 128, 0, 513]
    with Cache(qa, len(lens), 2 * hkv, hkv, d, 520) as c:
        c.fill(lens, 5)
        c.check_read(lens)
        c.check_read(lens, [10, 0, 62, 64, 63, 0, 0, 449], [50, 1, 1, 1, 66, 128, 0, 64])


@pytest.mark.parametrize("d", [64, 128])
def test_what_is_held_does_not_depend_on_the_calls(qa, d):
    lens, cuts = [300, 129, 64], [[1, 62, 1, 3, 61, 70, 102], [64, 64, 1], [63, 1]]
    k, v = rows(1, sum(lens), 2, d), rows(2, sum(lens), 2, d)
    offs = np.cumsum([0] + lens)
    with Cache(qa, 3, 4, 2, d, 320) as c:
        at = [0, 0, 0]
        for step in range(7):
            n = [cut[step] if step < len(cut) else 0 for cut in cuts]
            part = [x for b in range(3) for x in range(offs[b] + at[b], offs[b] + at[b] + n[b])]
            c.append(at, n, k[part].contiguous(), v[part].contiguous())
            at = [a + m for a, m in zip(at, n)]
            c.check_read(at)
        assert at == lens


@pytest.mark.parametrize("d", [64, 128])
def test_blocks_of_every_size_of_number(qa, d):
    """Largest magnitudes over bf16's range, ties, zeros, values below 2^-64, and some
    that are not finite: each in a block of its own."""
    rng = np.random.default_rng(d)
    tops = [2.0 ** e for e in range(-126, 127, 11)] + [0.0, 2.0 ** -64, 2.0 ** -65 * 1.9921875, 3.3895e38, 127.0, 254.0]
    x = rng.uniform(-1, 1, (len(tops) + 3, BLOCK, 1, d)).astype(np.float32)
    halves = (rng.integers(-126, 127, x.shape) + 0.5).astype(np.float32) / 127  # a tie where the scale is a power of two / 127
    x = np.where(rng.random(x.shape) < 0.5, x, halves)
    x[:, 5, 0, 3] = 1.0
    for i, top in enumerate(tops):
        x[i] *= np.float32(top)
    x[len(tops), 63, 0, d - 1] = np.nan
    x[len(tops) + 1, 0, 0, 0] = np.inf
    x[len(tops) + 2, 17, 0, 9] = -np.inf
    n = x.shape[0] * BLOCK
    k = torch.from_numpy(x.reshape(n, 1, d)).cuda().bfloat16()
    with Cache(qa, 1, 1, 1, d, n + 3) as c:
        c.append([0], [n], k, k.flip(0).contiguous())
        c.check_read([n])


def test_ranges_elsewhere_are_left_alone(qa):
    with Cache(qa, 3, 4, 2, 128, 256, layers=2) as c:
        c.fill([100, 256, 31], 3)
        k, v = rows(9, 5, 2, 128), rows(10, 5, 2, 128)
        qa.qa_q8_append(c.h, 1, [0, 0, 0], [2, 0, 3], k, v)  # another layer
        c.check_read([100, 256, 31])
        c.append([100, 0, 0], [5, 0, 0], k, v)  # sequences with nothing new
        c.check_read([105, 256, 31])
        ko = torch.zeros(5, 2, 128, device="cuda", dtype=torch.bfloat16)
        qa.qa_q8_read(c.h, 1, [0, 0, 0], [2, 0, 3], ko, None)
        assert torch.equal(ko, k)


# ------------------------------------------------------------------ decode
GEOMETRIES = [(1, 1, 64), (8, 1, 128), (4, 2, 64), (6, 6, 128), (16, 8, 128), (32, 8, 128), (32, 4, 64)]


@pytest.mark.parametrize("hq,hkv,d", GEOMETRIES)
def test_decode_is_attention_over_what_is_held(qa, hq, hkv, d):
    lens = [0, 1, 63, 64, 65, 127, 128, 700, 1500]
    with Cache(qa, len(lens), hq, hkv, d, 1600) as c:
        c.fill(lens, 11)
        q, k, v = c.tokens(len(lens), 21)
        out = torch.full_like(q, 9.0)
        kh, vh = torch.empty_like(k), torch.empty_like(v)
        qa.qa_q8_decode_step(c.h, 0, lens, q, k, v, None, None, out, kh, vh)
        assert torch.equal(kh, k) and torch.equal(vh, v)
        c.ref.write(lens, [1] * len(lens), f64(k), f64(v))
        for b, pos in enumerate(lens):
            close(out[b:b + 1], *c.want(b, pos, q[b:b + 1].double()), what=f"position {pos}")
        c.check_read([n + 1 for n in lens])
        assert qa.qa_q8_get_device_error(c.h)[0] == 0


@pytest.mark.parametrize("d", [64, 128])
def test_decode_steps_follow_each_other_through_blocks(qa, d):
    lens = [60, 126, 0]
    with Cache(qa, 3, 8, 2, d, 512) as c:
        c.fill(lens, 31)
        for step in range(70):
            q, k, v = c.tokens(3, 100 + 3 * step)
            out = torch.empty_like(q)
            qa.qa_q8_decode_step(c.h, 0, lens, q, k, v, None, None, out)
            c.ref.write(lens, [1, 1, 1], f64(k), f64(v))
            if step % 9 < 6:
                for b, pos in enumerate(lens):
                    close(out[b:b + 1], *c.want(b, pos, q[b:b + 1].double()), what=f"step {step}, position {pos}")
            lens = [n + 1 for n in lens]
        c.check_read(lens)
