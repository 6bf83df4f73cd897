"""Rows of the 4-bit cache that an attention window hides from a token reach none
of its outputs, whatever they hold (GPU).  Expected values and tolerances as in
test_gpu_q4.py."""
import pytest
import torch

from gpu_util import f64
from test_gpu_q4 import DECODE_BITS, Cache, close

pytestmark = pytest.mark.gpu
NAN = 0x7F


@pytest.fixture(scope="module")
def qa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gqa_attention_preallocated_qa_gb300 import _build
    _build.build()
    from gqa_attention_preallocated_qa_gb300 import binding
    return binding


def put_nan(c, b, row, kv, group):
    """Makes one group of a row (every kv head) NaN: in the cache, not in the copy."""
    c.views()[1 if kv == "k" else 3][b, :, row, group] = NAN


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 1, 64), (4, 4, 64), (4, 2, 128), (8, 1, 128)])
@pytest.mark.parametrize("ntok", [2, 5, 8, 16])
@pytest.mark.parametrize("kv", ["k", "v"])
@pytest.mark.parametrize("start,window", [(100, 40), (200, 70), (300, 264), (103, 40)])
def test_a_row_that_only_the_first_tokens_of_a_chunk_see(qa, hq, hkv, d, ntok, kv, start, window):
    # Token t at start + t sees rows from start + t + 1 - window on: row `row` is
    # seen by the tokens 0 .. half - 1 alone.
    half = max(1, min(ntok, 8) // 2)
    row, group = start - window + half, d // 32 - 1
    with Cache(qa, 1, 2, hq, hkv, d, start + 20) as c:
        qa.qa_q4_cache_set_window(c.h, 0, window)
        starts, n = [start, start], [ntok, ntok]
        c.fill(0, starts, 5)
        put_nan(c, 0, row, kv, group)
        q, k, v = c.tokens(n, 6)
        out = torch.empty_like(q)
        qa.qa_q4_prefill(c.h, 0, starts, n, q, k, v, c.wq, c.wk, out)
        assert qa.qa_q4_get_device_error(c.h) == (0, 0)
        assert qa.qa_q4_stats(c.h)["prefill_attn"] == 0
        qp, kp = c.transform(starts, n, q, k, v)
        c.note(0, starts, n, kp, f64(v))
        want, mag = c.want(starts, n, qp, window=window)
        nan = torch.isnan(out)
        dims = torch.zeros(d, dtype=torch.bool, device="cuda")
        dims[32 * group:] = True
        seen = dims if kv == "v" else torch.ones_like(dims)
        assert torch.equal(nan[:half], seen.expand(half, hq, d))
        assert not nan[half:].any()
        close(out[half:], want[half:], mag[half:], DECODE_BITS)
