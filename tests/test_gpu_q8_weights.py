"""Weights of very different size in one warp of a step on the 8-bit cache, against the
definition (q8_ref.py).

Tolerance, from the roundings alone.  A weight is rounded to fp16 relative to a reference
that leaves the warp's largest weight at 2^7 or more: 2^-11 of the weight, or 2^-25 (half of
the smallest step) where that is more, which is 2^-32 of the largest.  Scores, in units of
log2, are below 2^5 here: eight fp32 sums of terms up to three times that size (a code
carries 128 that is taken away again) move one by 8 * 3 * 2^5 * 2^-24 < 2^-14, so a weight by
2^-14.  Numerator and denominator use the same weights: 2 (2^-11 + 2^-14) sum p |v| +
2^-31 sum |v| / l, with l relative to the largest weight, and one rounding to bf16, 2^-8 |out|.
A value's code n carries 128 as well, whatever n is: a block's sum is of 64 products p s (n + 128),
at most 255 p s, and starts at -128 s times a sum of the 64 weights.  An fp32 sum of 64 terms in
any order is off by 64 * 2^-23 of the sum of their magnitudes: 2^-17 (255 + 128) s sum p, and with
s = a / 127, a the block's largest |v|, 3.02 * 2^-17 a of the block's share of the weights.
The weights of the rows held in bf16 are sums of two bf16 numbers, inside that.
"""
import math

import pytest
import torch

from gpu_util import f64
from test_gpu_q8 import BLOCK, Cache, qa, rows  # noqa: F401

pytestmark = pytest.mark.gpu

HQ, HKV = 4, 1


def check(qa, d, score, value, new, blocks=0):
    """A step behind len(score) keys of these scores (units of log2, for a query of one
    dimension), value[j] in every dimension of V; new: the new token's score and value."""
    pos = len(score)
    by = d ** 0.5 / math.log2(math.e) / 16  # keys score / 16, queries 16 in these units
    q = torch.zeros(1, HQ, d, device="cuda", dtype=torch.bfloat16)
    q[:, :, 0] = 16 * by ** 0.5
    scale = 16 * by / float(q[0, 0, 0])
    with Cache(qa, 1, HQ, HKV, d, pos + 64) as c:
        k = torch.zeros(pos + 1, HKV, d, device="cuda")
        k[:, 0, 0] = torch.tensor([*score, new[0]], device="cuda") * scale
        v = torch.tensor([*value, new[1]], device="cuda").view(-1, 1, 1).expand(-1, HKV, d).contiguous()
        k, v = k.bfloat16(), v.bfloat16()
        c.append([0], [pos], k[:pos].contiguous(), v[:pos].contiguous())
        out = torch.empty_like(q)
        args = (q, k[pos:].contiguous(), v[pos:].contiguous(), None, None, out)
        lists = torch.empty(1, HKV, max(blocks, 1), dtype=torch.int32, device="cuda")
        if blocks:
            qa.qa_q8_sparse_step(c.h, 0, [pos], blocks, *args, lists)
        else:
            qa.qa_q8_decode_step(c.h, 0, [pos], *args)
        c.ref.write([pos], [1], f64(k[pos:]), f64(v[pos:]))
        want, mag, flat = c.want(0, pos, q.double(), lists[0].cpu().numpy() if blocks else None)
        a = 127 * float(c.ref.s[1, 0, 0, :pos // BLOCK].max())
    close(out, want, mag, flat, a)


def close(out, want, mag, flat, a):
    tol = 2.0 ** -8 * want.abs() + 2 * (2.0 ** -11 + 2.0 ** -14) * mag + 2.0 ** -31 * flat + 3.02 * 2.0 ** -17 * a
    worst = float(((out.double() - want).abs() / tol).max())
    assert worst <= 1, f"{worst:.3f} of the tolerance: {float(out[0, 0, 0])} for {float(want[0, 0, 0])}"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("pos,at", [(256, 5), (256, 250), (300, 70), (20000, 9), (20000, 19000)])
@pytest.mark.parametrize("blocks", [0, 4])
def test_one_key_far_above_a_flat_tail(qa, d, pos, at, blocks):
    """2^26 times the weight of each other key, and a value of zero: the output is the tail's."""
    score, value = [0.0] * pos, [1.0] * pos
    score[at], value[at] = 26.0, 0.0
    check(qa, d, score, value, (0.0, 1.0), blocks)


@pytest.mark.parametrize("at", [9, 64 * 130])
def test_a_long_flat_tail_in_few_warps(qa, at):
    """The same where four warps take all keys of a kv head: a quarter of them share the warp of
    the key that is far above."""
    d, hkv, pos, far = 64, 304, 20000, 26.0
    by = d ** 0.5 / math.log2(math.e)
    q = torch.zeros(1, hkv, d, device="cuda", dtype=torch.bfloat16)
    q[:, :, 0] = 4 * by
    k = torch.zeros(pos + 1, hkv, d, device="cuda", dtype=torch.bfloat16)
    k[at, :, 0] = far / 4
    v = torch.ones_like(k)
    v[at] = 0
    h = qa.qa_q8_cache_alloc(1, 1, hkv, hkv, d, pos + 1)
    try:
        qa.qa_q8_append(h, 0, [0], [pos], k[:pos], v[:pos])
        out = torch.empty_like(q)
        qa.qa_q8_decode_step(h, 0, [pos], q, k[pos:], v[pos:], None, None, out)
    finally:
        qa.qa_q8_cache_free(h)
    # the key far above: its code is 127, s = (far / 4) / 127 in fp32
    t = float(q[0, 0, 0].double()) * 127 * float(k[at, 0, 0].float() / 127) * math.log2(math.e) / d ** 0.5
    tail = pos * 2.0 ** -t  # all but one key, and the new token
    want = torch.full((1, hkv, d), tail / (1 + tail), device="cuda", dtype=torch.float64)
    close(out, want, want, torch.full_like(want, pos / (1 + tail)), 1.0)


@pytest.mark.parametrize("d", [64, 128])
def test_the_new_token_far_above_what_is_held(qa, d):
    check(qa, d, [0.0] * 300, [1.0] * 300, (26.0, 0.0))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("span", [6.0, 14.5, 30.0])
def test_scores_over_the_whole_range(qa, d, span):
    gen = torch.Generator().manual_seed(int(span))
    pos = 9000
    score = (torch.rand(pos, generator=gen) * span).tolist()
    value = torch.randn(pos, generator=gen).tolist()
    check(qa, d, score, value, (1.0, 2.0))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("step", [0.11, 0.9])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_that_rise_and_fall_from_block_to_block(qa, d, step, sign):
    """The reference follows the scores of a warp's blocks up, in many small steps or a few
    large ones, or stays where the first one put it."""
    n = 280
    score = [sign * (step * (j // BLOCK) % 31.0 - 15.5) for j in range(n * BLOCK)]
    value = [1.0 + (j // BLOCK) % 5 for j in range(n * BLOCK)]
    check(qa, d, score, value, (0.0, -1.0))


@pytest.mark.parametrize("d", [64, 128])
def test_values_of_the_largest_size(qa, d):
    """Weights that grow to 2^15 times values near bf16's largest number."""
    n = 6
    score = [2.4 * (j // BLOCK) for j in range(n * BLOCK)]
    check(qa, d, score, [2.0 ** 126 * (1 if j % 3 else -1) for j in range(n * BLOCK)], (0.0, 2.0 ** 126))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [23, 24, 25, 26, 27, 28])
def test_scores_whose_steps_are_larger_than_one(qa, d, size):
    """Scores near 2^size differ between blocks by up to 32, in steps of fp32 there: the weights
    are what rounding leaves of them, and the outputs stay between the values."""
    n, batch = 48, 8
    gen = torch.Generator(device="cuda").manual_seed(size)
    with Cache(qa, batch, 8, 2, d, n * BLOCK + 10) as c:
        # dimension 0 has the score, dimension 1 what it differs by
        by = 2.0 ** size * d ** 0.5 / math.log2(math.e)
        q = torch.zeros(batch, 8, d, device="cuda")
        q[:, :, 0] = by ** 0.5
        q[:, :, 1] = by ** 0.5 * 2.0 ** (5 - size)
        k = torch.zeros(batch, n * BLOCK + 1, 2, d, device="cuda")
        k[..., 0] = by ** 0.5
        code = torch.randint(0, 128, (batch, n, 1, 2), generator=gen, device="cuda") / 127
        k[:, :-1, :, 1] = by ** 0.5 * code.expand(-1, -1, BLOCK, -1).reshape(batch, n * BLOCK, 2)
        v = 1 + torch.rand(k.shape, generator=gen, device="cuda")
        q, k, v = q.bfloat16(), k.bfloat16(), v.bfloat16()
        qa.qa_q8_append(c.h, 0, [0] * batch, [n * BLOCK] * batch, k[:, :-1].flatten(0, 1).contiguous(), v[:, :-1].flatten(0, 1).contiguous())
        out = torch.empty_like(q)
        qa.qa_q8_decode_step(c.h, 0, [n * BLOCK] * batch, q, k[:, -1].contiguous(), v[:, -1].contiguous(), None, None, out)
        assert torch.isfinite(out).all()
        assert float(out.min()) >= 1 - 2.0 ** -6 and float(out.max()) <= 2 + 2.0 ** -5
