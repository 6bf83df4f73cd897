"""What a 4-bit cache takes of the device's memory and when, and its rotary table
(GPU): the workspace and the sums of prefill attention come with the first call
that needs them, and caches share a table that the device computes."""
import numpy as np
import pytest
import torch

import q4_ref
from gpu_util import f64
from test_gpu_q4 import EPS, PREFILL_BITS, THETA, Cache, close, rows

pytestmark = pytest.mark.gpu
MB = 1 << 20


@pytest.fixture(scope="module")
def qa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gqa_attention_preallocated_qa_gb300 import _build
    _build.build()
    from gqa_attention_preallocated_qa_gb300 import binding
    return binding


def taken(free):
    torch.cuda.synchronize()
    return free - torch.cuda.mem_get_info()[0]


def test_only_a_prefill_that_needs_it_takes_the_workspace(qa):
    b, hkv, d, cap = 8, 8, 128, 65536
    n = [1] * b
    q, k, v = (rows(i, b * 40, hkv, d) for i in (1, 2, 3))
    w = torch.ones(d, device="cuda").bfloat16()
    out = torch.empty_like(q)
    workspace = 2 * b * hkv * cap * d * 2
    free = torch.cuda.mem_get_info()[0]
    h = qa.qa_q4_cache_alloc(1, b, hkv, hkv, d, cap, THETA, EPS)
    try:
        held, scratch = qa.qa_q4_memory_info(h)
        table = cap * (d // 2) * 8
        assert scratch >= workspace + table
        qa.qa_q4_append(h, 0, [0] * b, n, k, v)
        qa.qa_q4_read(h, 0, [0] * b, n, q, out)
        qa.qa_q4_decode_step(h, 0, n, q, k, v, w, w, out)
        qa.qa_q4_prefill(h, 0, [2] * b, [16] * b, q, k, v, w, w, out)  # few tokens: the decode kernel
        assert taken(free) <= held + table + 32 * MB < workspace
        qa.qa_q4_prefill(h, 0, [18] * b, [40] * b, q, k, v, w, w, out)
        assert workspace <= taken(free) <= held + scratch + 32 * MB
        assert qa.qa_q4_get_device_error(h) == (0, 0)
    finally:
        qa.qa_q4_cache_free(h)
    assert taken(free) <= 32 * MB


def test_caches_share_a_rotary_table(qa):
    cap, d = 1 << 20, 128
    table = cap * (d // 2) * 8
    free = torch.cuda.mem_get_info()[0]
    a = qa.qa_q4_cache_alloc(1, 1, 1, 1, d, cap, THETA, EPS)
    one = taken(free)
    shorter = qa.qa_q4_cache_alloc(2, 1, 1, 1, d, cap // 2, THETA, EPS)
    other = qa.qa_q4_cache_alloc(1, 1, 1, 1, d, cap // 4, 2 * THETA, EPS)  # another base: a table of its own
    held = qa.qa_q4_memory_info(shorter)[0] + qa.qa_q4_memory_info(other)[0]
    assert one >= table
    assert table // 4 <= taken(free) - one - held <= table // 4 + 32 * MB
    qa.qa_q4_cache_free(a)      # `shorter` still reads the table
    assert taken(free) >= table
    n = 20
    k, v = rows(1, n, 1, d), rows(2, n, 1, d)
    q, w = rows(3, n, 1, d), torch.ones(d, device="cuda").bfloat16()
    outs = [torch.empty_like(q) for _ in range(2)]
    try:
        qa.qa_q4_prefill(shorter, 0, [0], [n], q, k, v, w, w, outs[0])
        fresh = qa.qa_q4_cache_alloc(1, 1, 1, 1, d, 64, THETA, EPS)
        qa.qa_q4_prefill(fresh, 0, [0], [n], q, k, v, w, w, outs[1])
        assert qa.qa_q4_get_device_error(fresh) == (0, 0)
        qa.qa_q4_cache_free(fresh)
        assert torch.equal(*outs)
    finally:
        qa.qa_q4_cache_free(shorter)
        qa.qa_q4_cache_free(other)
    assert taken(free) <= 32 * MB


@pytest.mark.parametrize("d", [64, 128])
def test_the_table_is_the_bf16_caches(qa, d):
    # The bf16 cache computes its table on the host.  Keys rotated at near and far
    # positions through either quantise to the same bytes: the tables agree within
    # a bit of fp32, which is 2^-16 of a step of the bf16 rounding behind them.
    start, ntok = [0, 70001, 149000], [200] * 3
    with Cache(qa, 1, 3, 4, 2, d, 149200) as c:
        q, k, v = c.tokens(ntok, 4)
        qa.qa_q4_prefill(c.h, 0, start, ntok, q, k, v, c.wq, c.wk, torch.empty_like(q))
        assert qa.qa_q4_get_device_error(c.h) == (0, 0)
        _, kp = c.transform(start, ntok, q, k, v)
        kr, vr = torch.empty_like(k), torch.empty_like(v)
        qa.qa_q4_read(c.h, 0, start, ntok, kr, vr)
        np.testing.assert_array_equal(f64(kr), q4_ref.values(*q4_ref.quantise(kp)))
        np.testing.assert_array_equal(f64(vr), q4_ref.values(*q4_ref.quantise(f64(v))))


def test_the_first_prefill_beside_a_capture(qa):
    # It allocates the workspace; a capture under way on another stream goes on.
    ntok = [60, 41]
    with Cache(qa, 1, 2, 8, 2, 128, 64) as c:
        q, k, v = c.tokens(ntok, 6)
        out = torch.empty_like(q)
        x = torch.zeros(64, device="cuda")
        torch.cuda.synchronize()
        graph, side, mine = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.stream(side):
            graph.capture_begin()
            try:
                x.add_(1)
                qa.qa_q4_prefill(c.h, 0, [0, 0], ntok, q, k, v, c.wq, c.wk, out, stream=mine)
            finally:
                graph.capture_end()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert (x == 1).all()
        qp, kp = c.transform([0, 0], ntok, q, k, v)
        c.note(0, [0, 0], ntok, kp, f64(v))
        c.check_bytes()
        want, mag = c.want([0, 0], ntok, qp)
        close(out, want, mag, PREFILL_BITS)


def test_a_captured_prefill_is_refused_before_it_allocates(qa):
    b, hkv, d, cap = 8, 8, 128, 16384
    q, k, v = (rows(i, b * 40, hkv, d) for i in (1, 2, 3))
    w, out = torch.ones(d, device="cuda").bfloat16(), torch.empty_like(q)
    h = qa.qa_q4_cache_alloc(1, b, hkv, hkv, d, cap, THETA, EPS)
    try:
        free = torch.cuda.mem_get_info()[0]
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.capture_begin()
            try:
                out.add_(0)
                with pytest.raises(qa.QaError) as e:
                    qa.qa_q4_prefill(h, 0, [0] * b, [40] * b, q, k, v, w, w, out, stream=side)
            finally:
                graph.capture_end()
        assert e.value.status == 5
        assert taken(free) <= 32 * MB
        assert qa.qa_q4_stats(h)["prefill_attn"] == 0
    finally:
        qa.qa_q4_cache_free(h)
