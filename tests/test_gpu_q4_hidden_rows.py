"""Rows of the 4-bit cache that an attention window hides from a token reach none
of its outputs, whatever they hold (GPU).  Expected values and tolerances as in
test_gpu_q4.py."""
import pytest
import torch

from gpu_util import f64
from test_gpu_q4 import DECODE_BITS, PREFILL_BITS, Cache, close

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


@pytest.mark.parametrize("hq,hkv,d,start,ntok,window", [
    (8, 2, 128, [300, 140], [200, 77], 150),
    (32, 8, 128, [1000] * 4, [300, 140, 129, 400], 200),
    (16, 8, 64, [900, 700], [300, 40], 170),
    (8, 2, 128, [5000], [100], 3000),          # keys in parts
    (24, 3, 128, [500, 90], [60, 200], 130),   # the transform kernel and a quantiser after it
])
@pytest.mark.parametrize("kv", ["k", "v"])
def test_rows_below_every_window_of_a_prefill(qa, hq, hkv, d, start, ntok, window, kv):
    # They may never have been written: NaN scales up to the row before the first
    # token's window, which lies inside a tile of 128 keys.
    with Cache(qa, 1, len(start), hq, hkv, d, max(s + n for s, n in zip(start, ntok))) as c:
        qa.qa_q4_cache_set_window(c.h, 0, window)
        c.fill(0, start, 5)
        for b, s in enumerate(start):
            for i in ((1,) if kv == "k" else (3,)):
                c.views()[i][b, :, :max(0, s + 1 - window)] = NAN
        q, k, v = c.tokens(ntok, 6)
        out = torch.empty_like(q)
        qa.qa_q4_prefill(c.h, 0, start, ntok, q, k, v, c.wq, c.wk, out)
        assert qa.qa_q4_get_device_error(c.h) == (0, 0)
        assert qa.qa_q4_stats(c.h)["prefill_attn"] > 0
        qp, kp = c.transform(start, ntok, q, k, v)
        c.note(0, start, ntok, kp, f64(v))
        want, mag = c.want(start, ntok, qp, window=window)
        close(out, want, mag, PREFILL_BITS)
