"""Which kernels the calls of the 4-bit cache take, on the GPU: the prefill form of
geometries whose token does not fit the row kernel's stages (the transform kernel
and a quantiser in place after it), and the border between the decode and the
prefill kernel.  Expected values and tolerances as in test_gpu_q4.py."""
import pytest
import torch

from gpu_util import f64
from test_gpu_q4 import DECODE_BITS, PREFILL_BITS, Cache, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gqa_attention_preallocated_qa_gb300 import _build
    _build.build()
    from gqa_attention_preallocated_qa_gb300 import binding
    return binding


def prefill_and_check(qa, c, start, ntok, window=0, seed=6):
    """One prefill of the cache c: bytes written, outputs and the error word."""
    q, k, v = c.tokens(ntok, seed)
    out = torch.full_like(q, float("nan"))
    qa.qa_q4_prefill(c.h, 0, start, ntok, q, k, v, c.wq, c.wk, out)
    assert qa.qa_q4_get_device_error(c.h) == (0, 0)
    # The reference's q' and k' come from the same transform kernel on the bf16
    # cache, so the bytes are equal, whatever its order of summation.
    qp, kp = c.transform(start, ntok, q, k, v)
    c.note(0, start, ntok, kp, f64(v))
    c.check_bytes()
    want, mag = c.want(start, ntok, qp, window=window)
    return out, want, mag


@pytest.mark.parametrize("hq,hkv,d,start,ntok,window", [
    (24, 3, 128, [0], [40], 0),
    (24, 3, 128, [0, 300, 17], [129, 77, 260], 0),
    (20, 5, 128, [700, 0, 90], [60, 200, 0], 0),
    (24, 3, 128, [1000, 300, 5], [150, 90, 200], 260),          # older rows from the window's tile on
    (24, 3, 128, [31] * 11, [20, 0, 3, 150, 9, 1, 20, 33, 128, 2, 17], 0),  # two groups of sequences, some in K5
    (24, 3, 128, [6000], [100], 0),                              # keys in parts
    (48, 6, 128, [5000, 0], [40, 130], 3000),
    (160, 160, 128, [0, 40], [33, 20], 0),                       # no number of shares fits
    (512, 64, 128, [20], [17], 0),
])
def test_prefill_of_tokens_too_wide_for_the_row_kernel(qa, hq, hkv, d, start, ntok, window):
    with Cache(qa, 1, len(start), hq, hkv, d, max(s + n for s, n in zip(start, ntok))) as c:
        qa.qa_q4_cache_set_window(c.h, 0, window)
        c.fill(0, start, 5)
        appended = qa.qa_q4_stats(c.h)["quantise"]
        out, want, mag = prefill_and_check(qa, c, start, ntok, window)
        stats = qa.qa_q4_stats(c.h)
        assert stats["norm_rope"] == stats["prefill_attn"] == stats["quantise"] - appended >= 1
        close(out, want, mag, PREFILL_BITS)


def test_wide_tokens_in_chunks_then_a_decode_step(qa):
    # A prompt, a chunk behind it through the same form, and a step over both.
    with Cache(qa, 1, 2, 24, 3, 128, 400) as c:
        for start, ntok in (([0, 0], [150, 60]), ([150, 60], [90, 200])):
            out, want, mag = prefill_and_check(qa, c, start, ntok, seed=start[0] + 7)
            close(out, want, mag, PREFILL_BITS)
        at, one = [240, 260], [1, 1]
        q, k, v = c.tokens(one, 9)
        out = torch.empty_like(q)
        qa.qa_q4_decode_step(c.h, 0, at, q, k, v, c.wq, c.wk, out)
        qp, kp = c.transform(at, one, q, k, v)
        c.note(0, at, one, kp, f64(v))
        c.check_bytes()
        want, mag = c.want(at, one, qp)
        close(out, want, mag, DECODE_BITS)


@pytest.mark.parametrize("start,ntok,window,decode", [
    (0, 16, 0, 2), (0, 17, 0, 0),
    (511, 16, 0, 2), (511, 17, 0, 0),
    (512, 17, 0, 3), (512, 24, 0, 3), (512, 25, 0, 0),
    (5000, 24, 0, 3), (5000, 25, 0, 0),
    (5000, 16, 511, 2), (5000, 17, 511, 0),      # a window below 512 keys counts, not the cache
    (5000, 24, 512, 3), (5000, 25, 512, 0),
])
def test_the_border_between_the_two_kernels(qa, start, ntok, window, decode):
    # decode: launches of eight tokens; 0: the prefill kernel.
    with Cache(qa, 1, 1, 8, 2, 128, start + ntok) as c:
        qa.qa_q4_cache_set_window(c.h, 0, window)
        c.fill(0, [start], 5)
        out, want, mag = prefill_and_check(qa, c, [start], [ntok], window)
        stats = qa.qa_q4_stats(c.h)
        assert (stats["decode"], stats["prefill_attn"]) == (decode, 0 if decode else 1)
        close(out, want, mag, DECODE_BITS if decode else PREFILL_BITS)


@pytest.mark.parametrize("ntok", [1, 4, 16, 17])
def test_an_output_copied_into_the_next_calls_inputs(qa, ntok):
    # A chain of calls, each one's queries, keys and values made of the last one's
    # outputs by kernels in between, with nothing else that waits: the same bits as
    # with a synchronisation after every call.
    layers, n = 3, [ntok, ntok]
    with Cache(qa, layers, 2, 8, 2, 128, 700 + 6 * ntok) as c:
        q0, k0, v0 = c.tokens(n, 6)
        got = []
        for wait in (False, True):
            for layer in range(layers):
                c.fill(layer, [600, 600], 5)
            q, k, v, out = q0.clone(), k0.clone(), v0.clone(), torch.empty_like(q0)
            outs = []
            torch.cuda.synchronize()
            for i in range(6):
                for layer in range(layers):
                    at = [600 + i * ntok] * 2
                    if ntok == 1:
                        qa.qa_q4_decode_step(c.h, layer, at, q, k, v, c.wq, c.wk, out)
                    else:
                        qa.qa_q4_prefill(c.h, layer, at, n, q, k, v, c.wq, c.wk, out)
                    q.copy_(out)
                    k.copy_(out[:, :2])
                    v.copy_(out[:, 2:4])
                    outs.append(out.clone())
                    if wait:
                        torch.cuda.synchronize()
            got.append(outs)
        assert qa.qa_q4_get_device_error(c.h) == (0, 0)
        assert all(torch.equal(a, b) for a, b in zip(*got))
