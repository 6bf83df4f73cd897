"""Forms of the 8-bit cache's steps beside those of test_gpu_q8.py: sparse steps with norm and
rotation, dense steps over caches that sixteen thread blocks share and that one has alone, and
rows that are not finite in the block being filled."""
import numpy as np
import pytest
import torch

import q8_ref
from gpu_util import f64
from test_gpu_q8 import BLOCK, Cache, close, qa, rows, transform  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ norm and rotation
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 128), (8, 1, 128), (8, 1, 64), (32, 8, 128), (8, 4, 64)])
@pytest.mark.parametrize("n_blocks", [2, 5])
def test_sparse_step_norms_and_rotates_before_it_chooses(qa, hq, hkv, d, n_blocks):
    """Raw rows and weights: the lists and outputs of the normed, rotated queries.  Sequences
    of one thread block and of several, and of nothing to choose."""
    lens = [0, 63, 130, 700, 2047, 3000]
    with Cache(qa, len(lens), hq, hkv, d, 3100) as c:
        c.fill(lens, 7)
        # (weights far from 1, so that raw queries would choose otherwise)
        c.wq, c.wk = rows(91, d), rows(92, d)
        for step in range(2):
            q, k, v = c.tokens(len(lens), 70 + 3 * step)
            q = q * torch.linspace(0.1, 4, hq, device="cuda", dtype=torch.bfloat16)[:, None]  # heads of different size
            qp, kp = transform(qa, c, lens, [1] * len(lens), q, k, v)
            out, kh, vh = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
            lists = torch.full((len(lens), hkv, n_blocks), 12345, device="cuda", dtype=torch.int32)
            qa.qa_q8_sparse_step(c.h, 0, lens, n_blocks, q, k, v, c.wq, c.wk, out, lists, kh, vh)
            assert torch.equal(kh, kp) and torch.equal(vh, v)
            c.ref.write(lens, [1] * len(lens), f64(kp), f64(v))
            got, g, other = lists.cpu().numpy(), hq // hkv, 0
            for b, pos in enumerate(lens):
                full = pos // BLOCK
                for h in range(hkv):
                    held = c.ref.n[0, b, h, :full], c.ref.s[0, b, h, :full]
                    want = q8_ref.select(f64(qp[b, h * g:(h + 1) * g]), *held, n_blocks)
                    np.testing.assert_array_equal(got[b, h], want, err_msg=f"position {pos}, kv head {h}")
                    other += (want != q8_ref.select(f64(q[b, h * g:(h + 1) * g]), *held, n_blocks)).any()
                close(out[b:b + 1], *c.want(b, pos, qp[b:b + 1].double(), got[b]), what=f"position {pos}")
            assert other > 0 or n_blocks == 2  # (two are the first and the last, whatever the queries)
            lens = [n + 1 for n in lens]


# ------------------------------------------------------------------ dense steps over long caches
@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (4, 2, 64), (2, 2, 128)])
def test_dense_step_over_many_blocks(qa, hq, hkv, d):
    """Sixteen thread blocks of many blocks each, and sequences of a few beside them."""
    lens = [60000, 33333, 4096, 100]
    with Cache(qa, 4, hq, hkv, d, 60100) as c:
        c.fill(lens, 11)
        for normed in (False, True):
            q, k, v = c.tokens(4, 21)
            qp, kp = transform(qa, c, lens, [1] * 4, q, k, v) if normed else (q, k)
            out = torch.empty_like(q)
            qa.qa_q8_decode_step(c.h, 0, lens, q, k, v, *((c.wq, c.wk) if normed else (None, None)), out)
            c.ref.write(lens, [1] * 4, f64(kp), f64(v))
            for b, pos in enumerate(lens):
                close(out[b:b + 1], *c.want(b, pos, qp[b:b + 1].double()), what=f"position {pos}")
            lens = [n + 1 for n in lens]
        assert qa.qa_q8_get_device_error(c.h)[0] == 0


@pytest.mark.parametrize("d", [64, 128])
def test_dense_step_with_more_sequences_than_sms(qa, d):
    """One thread block a sequence and kv head, many blocks each."""
    n, hkv = 40, 8
    lens = [300 + (739 * i) % 2700 for i in range(n)]
    with Cache(qa, n, hkv, hkv, d, 3100) as c:
        c.fill(lens, 11)
        q, k, v = c.tokens(n, 21)
        out = torch.empty_like(q)
        qa.qa_q8_decode_step(c.h, 0, lens, q, k, v, None, None, out)
        c.ref.write(lens, [1] * n, f64(k), f64(v))
        for b in range(0, n, 3):
            close(out[b:b + 1], *c.want(b, lens[b], q[b:b + 1].double()), what=f"position {lens[b]}")


# ------------------------------------------------------------------ rows that are not finite
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("new", [False, True])
def test_a_value_that_is_not_finite_in_the_block_being_filled(qa, d, bad, new):
    """In a row of V, of the cache or of the step: its dimension of its kv head's queries is
    not finite, and nothing else."""
    with Cache(qa, 1, 8, 2, d, 400) as c:
        c.fill([300], 3)
        q, k, v = c.tokens(1, 8)
        vs = rows(9, 5, 2, d)
        (v if new else vs)[0, 1, 7] = bad
        qa.qa_q8_append(c.h, 0, [300], [5], rows(10, 5, 2, d), vs)
        out = torch.empty_like(q)
        qa.qa_q8_decode_step(c.h, 0, [305], q, k, v, None, None, out)
        odd = ~torch.isfinite(out[0])
        assert odd[4:, 7].all() and odd.sum() == 4
