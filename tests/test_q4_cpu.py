"""The 4-bit format's reference against brute force, and the refusals of
qa_q4_* that need no device (nothing is launched here)."""
import ctypes

import numpy as np
import pytest

import q4_ref
from gqa_attention_preallocated_qa_gb300.inputs import bf16_bits_to_f64


@pytest.fixture(scope="module")
def qa():
    from gqa_attention_preallocated_qa_gb300 import _build
    _build.build()
    from gqa_attention_preallocated_qa_gb300 import binding
    return binding


def test_scales_are_the_upper_bytes_of_fp16():
    half = (np.arange(0x54, dtype=np.uint16) << 8).view(np.float16).astype(np.float64)
    np.testing.assert_array_equal(q4_ref.SCALES, half)
    assert q4_ref.SCALES.max() == 56 and (np.diff(q4_ref.SCALES) > 0).all()


def test_values_fit_bf16_exactly():
    codes = np.arange(256, dtype=np.uint8)[None, :16].repeat(0x54, 0)
    codes[:] = (np.arange(16) * 17)[None]
    v = q4_ref.values(codes, np.arange(0x54, dtype=np.uint8)[:, None])
    f = v.astype(np.float32)
    assert (f == v).all() and not (f.view(np.uint32) & 0xFFFF).any()


def test_quantiser_rounds_to_nearest():
    rng = np.random.default_rng(0)
    x = bf16_bits_to_f64(rng.integers(0, 0x4380, (500, 128)).astype(np.uint16) | (rng.integers(0, 2, (500, 128)) << 15).astype(np.uint16))
    codes, scales = q4_ref.quantise(x)
    v = q4_ref.values(codes, scales)
    s = q4_ref.SCALES[scales].repeat(32, -1)
    top = np.abs(x.reshape(500, 4, 32)).max(-1).repeat(32, -1)
    np.testing.assert_array_equal(np.abs(s - top / 7), np.abs(q4_ref.SCALES[:, None, None] - top / 7).min(0))
    inside = (x <= 7.5 * s) & (x >= -8.5 * s)
    assert (np.abs(x - v) <= 0.5 * s + 1e-300)[inside].all()


def test_null_cache_is_rejected_everywhere(qa):
    lens = (ctypes.c_int32 * 1)(4)
    lib = qa.lib
    assert lib.qa_q4_cache_alloc(None, None) == 1
    assert lib.qa_q4_cache_free(None) == 0
    assert lib.qa_q4_cache_set_window(None, 0, 0) == 1
    assert lib.qa_q4_append(None, 0, 1, lens, lens, 16, 16, None, None, None) == 1
    assert lib.qa_q4_read(None, 0, 1, lens, lens, 16, 16, None) == 1
    assert lib.qa_q4_prefill(None, 0, 1, lens, lens, 16, 16, 16, 16, 16, 16, None) == 1
    assert lib.qa_q4_decode_step(None, 0, 1, lens, 16, 16, 16, 16, 16, 16, None, None, None) == 1
    assert lib.qa_q4_decode_step_device_positions(None, 0, 1, 16, 16, 16, 16, 16, 16, 16, None, None, None) == 1
    assert lib.qa_q4_cache_view(None, 0, None, None, None, None, None) == 1
    assert lib.qa_q4_get_device_error(None, None) == 1
    assert lib.qa_q4_stats(None, None) == 1
    assert lib.qa_q4_memory_info(None, None, None) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=96), 2), (dict(n_q_heads=6, n_kv_heads=4), 2), (dict(n_q_heads=32, n_kv_heads=2), 2),
    (dict(capacity=0), 1), (dict(max_batch=0), 1), (dict(num_layers=0), 1), (dict(capacity=(1 << 24) + 1), 2),
    (dict(rope_theta=0.0), 1), (dict(rms_eps=-1.0), 1)])
def test_alloc_rejects_bad_geometry(qa, kw, status):
    args = dict(num_layers=1, max_batch=1, n_q_heads=32, n_kv_heads=8, head_dim=128, capacity=64,
                rope_theta=1e6, rms_eps=1e-6)
    args.update(kw)
    with pytest.raises(qa.QaError) as e:
        qa.qa_q4_cache_alloc(**args)
    assert e.value.status == status


def test_ranges_need_one_entry_per_sequence(qa):
    with pytest.raises(ValueError):
        qa.qa_q4_append(None, 0, [0, 0], [1], 16, 16)


def test_arguments_of_the_native_calls(qa):
    """Tensors, addresses, None; lists, tuples, int32 buffers: all reach the C
    entry point (which refuses the null cache), and nothing else does."""
    import torch
    x = torch.zeros(16, dtype=torch.bfloat16)
    for pos in ([0, 0], (0, 0), (ctypes.c_int32 * 2)(0, 0), np.zeros(2, np.int32), np.zeros(2, np.int64),
                torch.zeros(2, dtype=torch.int32)):
        with pytest.raises(qa.QaError) as e:
            qa.qa_q4_decode_step(None, 0, pos, x, x.data_ptr(), x, x, x, x, stream=0)
        assert e.value.status == 1
    for bad in ([0.5], ["0"], 3, None, [None]):
        with pytest.raises(TypeError):
            qa.qa_q4_decode_step(None, 0, bad, x, x, x, x, x, x, stream=0)
    with pytest.raises(OverflowError):
        qa.qa_q4_decode_step(None, 0, [1 << 31], x, x, x, x, x, x, stream=0)
    with pytest.raises(AttributeError):  # not a tensor
        qa.qa_q4_read(None, 0, [0], [1], np.zeros(4, np.uint16), x, stream=0)
    with pytest.raises(TypeError):
        qa._q4calls.read(None, 0, [0], [1])
