"""Sparse steps on caches of a long capacity: their shared memory goes by the sequences of the
launch (host positions) or by the capacity (device positions)."""
import pytest
import torch

import q8_ref
from gpu_util import f64
from test_gpu_q8 import BLOCK, Cache, check_sparse, close, qa  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (2, 2, 64)])
def test_short_sequences_in_a_long_cache(qa, hq, hkv, d):
    cap, lens, n_blocks = 1 << 20, [5000, 900, 64, 63], 6
    with Cache(qa, 4, hq, hkv, d, 6000) as c:  # the reference's capacity
        qa.qa_q8_cache_free(c.h)
        c.h = qa.qa_q8_cache_alloc(1, 4, hq, hkv, d, cap)
        c.fill(lens, 3)
        for i in range(2):
            lens = check_sparse(qa, c, lens, n_blocks, 40 + 3 * i)
        # one that has nothing to choose, and fewer sequences
        assert check_sparse(qa, c, [5002, 902], 79, 50) == [5003, 903]
        for dev in (True, False):
            q, k, v = c.tokens(4, 60)
            at = [5003, 903, 66, 65]
            out = torch.empty_like(q)
            lists = torch.empty(4, hkv, n_blocks, device="cuda", dtype=torch.int32)
            if dev:
                pos = torch.tensor(at, device="cuda", dtype=torch.int32)
                qa.qa_q8_sparse_step_device_positions(c.h, 0, 4, pos, n_blocks, q, k, v, None, None, out, lists)
            else:
                qa.qa_q8_sparse_step(c.h, 0, at, n_blocks, q, k, v, None, None, out, lists)
            c.ref.write(at, [1] * 4, f64(k), f64(v))
            for b, p in enumerate(at):
                got = lists[b].cpu().numpy()
                for h in range(hkv):
                    full = p // BLOCK
                    g = hq // hkv
                    want = q8_ref.select(f64(q[b, h * g:(h + 1) * g]), c.ref.n[0, b, h, :full], c.ref.s[0, b, h, :full], n_blocks)
                    assert (got[h] == want).all(), (dev, b, h)
                close(out[b:b + 1], *c.want(b, p, q[b:b + 1].double(), got), what=f"{dev}: position {p}")
        assert qa.qa_q8_get_device_error(c.h)[0] == 0
