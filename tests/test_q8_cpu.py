"""The 8-bit format's reference against brute force, and the refusals of
qa_q8_* that need no device (nothing is launched here)."""
import ctypes

import numpy as np
import pytest
import torch

import q8_ref


@pytest.fixture(scope="module")
def qa():
    from gqa_attention_preallocated_qa_gb300 import _build
    _build.build()
    from gqa_attention_preallocated_qa_gb300 import binding
    return binding


def blocks(seed, n, d):
    x = torch.randn(n, 64, d, generator=torch.Generator().manual_seed(seed)) * torch.logspace(-8, 8, n)[:, None, None]
    return x.bfloat16().float().numpy()


def test_quantiser_rounds_to_the_nearest_step():
    x = blocks(0, 20, 64)
    n, s = q8_ref.quantise(x)
    assert np.abs(n).max() == 127 and (np.abs(n).max((1, 2)) == 127).all()
    step = np.abs(x).max((1, 2)).astype(np.float64) / 127
    # half a step, and the roundings of the two quotients and the product to fp32
    assert (np.abs(x - q8_ref.values(n, s)) <= (0.5 + 127 * 2.0 ** -22) * step[:, None, None]).all()
    assert (np.abs(s - step) <= 2.0 ** -24 * step).all()


def test_blocks_of_nothing_and_of_nan():
    x = blocks(1, 4, 64)
    x[0] = 0
    x[1] = np.float32(2.0 ** -65)
    x[2, 3, 4] = np.inf
    n, s = q8_ref.quantise(x)
    assert (n[:3] == 0).all() and s[0] == 0 and s[1] == 0 and np.isnan(s[2]) and s[3] > 0


def test_scores_bound_the_products():
    """No product of the group's integers with a key passes its block's score."""
    rng = np.random.default_rng(2)
    n, s = q8_ref.quantise(blocks(3, 8, 64) * 1e-3)
    q = rng.standard_normal((4, 64)).astype(np.float32)
    c, _ = q8_ref._codes(q, (0, 1))
    score = q8_ref.scores(q, n, s)
    assert np.isinf(score[[0, -1]]).all()
    for j in range(1, 7):
        most = np.maximum((c[None] @ n[j].T)[0], 0).max()
        assert score[j] >= np.float32(most) * s[j] * (1 - 2.0 ** -23)
        assert (np.einsum("gd,kd->k", c, n[j]).max() * float(s[j])) <= score[j] * (1 + 2.0 ** -23)


def test_choice_takes_the_lower_index_among_equals():
    n, s = q8_ref.quantise(np.repeat(blocks(4, 1, 64), 9, 0))
    q = np.ones((2, 64), np.float32)
    assert q8_ref.select(q, n, s, 4).tolist() == [0, 1, 2, 8]
    assert q8_ref.select(q, n, s, 12).tolist() == [*range(9), -1, -1, -1]
    assert q8_ref.select(q, n[:0], s[:0], 2).tolist() == [-1, -1]


def test_attention_reference_by_hand():
    q = torch.tensor([[[1.0, 0.0]], [[0.0, 2.0]]]).double()
    k = torch.tensor([[[0.0, 0.0], [1.0, 1.0], [3.0, -1.0]]]).double()
    v = torch.tensor([[[1.0, 0.0], [0.0, 1.0], [5.0, 5.0]]]).double()
    out, mag, flat = q8_ref.attend(q, k, v, 1)
    w = torch.exp(torch.tensor([0.0, 1 / 2 ** 0.5]).double())
    torch.testing.assert_close(out[0, 0], w / w.sum())
    w = torch.exp(torch.tensor([0.0, 2 / 2 ** 0.5, -2 / 2 ** 0.5]).double())
    torch.testing.assert_close(out[1, 0], (w[:, None] * v[0]).sum(0) / w.sum())
    torch.testing.assert_close(mag, out)
    assert (flat >= mag).all()


def test_null_cache_is_rejected_everywhere(qa):
    lens = (ctypes.c_int32 * 1)(4)
    lib = qa.lib
    assert lib.qa_q8_cache_alloc(None, None) == 1
    assert lib.qa_q8_cache_free(None) == 0
    assert lib.qa_q8_append(None, 0, 1, lens, lens, 16, 16, None) == 1
    assert lib.qa_q8_read(None, 0, 1, lens, lens, 16, 16, None) == 1
    assert lib.qa_q8_prefill(None, 0, 1, lens, lens, 16, 16, 16, 16, 16, 16, None) == 1
    assert lib.qa_q8_decode_step(None, 0, 1, lens, 16, 16, 16, 16, 16, 16, None, None, None) == 1
    assert lib.qa_q8_decode_step_device_positions(None, 0, 1, 16, 16, 16, 16, 16, 16, 16, None, None, None) == 1
    assert lib.qa_q8_sparse_step(None, 0, 1, lens, 1, 16, 16, 16, 16, 16, 16, 16, None, None, None) == 1
    assert lib.qa_q8_sparse_step_device_positions(None, 0, 1, 16, 1, 16, 16, 16, 16, 16, 16, 16, None, None, None) == 1
    assert lib.qa_q8_get_device_error(None, None) == 1
    assert lib.qa_q8_stats(None, None) == 1
    assert lib.qa_q8_memory_info(None, None, None) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=96), 2), (dict(n_q_heads=6, n_kv_heads=4), 2), (dict(n_q_heads=32, n_kv_heads=2), 2),
    (dict(capacity=0), 1), (dict(max_batch=0), 1), (dict(num_layers=0), 1), (dict(capacity=(1 << 20) + 1), 2),
    (dict(rope_theta=0.0), 1), (dict(rms_eps=-1.0), 1), (dict(max_batch=65536), 2)])
def test_alloc_rejects_bad_geometry(qa, kw, status):
    args = dict(num_layers=1, max_batch=1, n_q_heads=32, n_kv_heads=8, head_dim=128, capacity=64,
                rope_theta=1e6, rms_eps=1e-6)
    args.update(kw)
    with pytest.raises(qa.QaError) as e:
        qa.qa_q8_cache_alloc(**args)
    assert e.value.status == status


@pytest.mark.parametrize("kw", [dict(max_batch=65535, n_q_heads=65535, n_kv_heads=65535, capacity=1 << 20),
                                dict(max_batch=65535, n_q_heads=8192, n_kv_heads=8192, capacity=128)])
def test_alloc_rejects_what_64_bits_cannot_count(qa, kw):
    """The second one's bytes would wrap: 2^31 - 1 layers of 2^30 blocks (less 2^14) of 16 KB."""
    with pytest.raises(qa.QaError) as e:
        qa.qa_q8_cache_alloc(**{**dict(num_layers=(1 << 31) - 1, head_dim=128, rope_theta=1e6, rms_eps=1e-6), **kw})
    assert e.value.status == 2


def test_arguments_of_the_native_calls(qa):
    """Tensors, addresses, None; lists, tuples, int32 buffers: all reach the C
    entry point (which refuses the null cache), and nothing else does."""
    x = torch.zeros(16, dtype=torch.bfloat16)
    for pos in ([0, 0], (0, 0), (ctypes.c_int32 * 2)(0, 0), np.zeros(2, np.int32), torch.zeros(2, dtype=torch.int32)):
        with pytest.raises(qa.QaError) as e:
            qa.qa_q8_decode_step(None, 0, pos, x, x.data_ptr(), x, None, None, x, stream=0)
        assert e.value.status == 1
        with pytest.raises(qa.QaError) as e:
            qa.qa_q8_sparse_step(None, 0, pos, 3, x, x.data_ptr(), x, x, x, x, x, stream=0)
        assert e.value.status == 1
    for call in (lambda: qa.qa_q8_append(None, 0, [0], [1], x, x, stream=0),
                 lambda: qa.qa_q8_read(None, 0, [0], [1], x, None, stream=0),
                 lambda: qa.qa_q8_prefill(None, 0, [0], [1], x, x, x, x, x, x, stream=0),
                 lambda: qa.qa_q8_decode_step_device_positions(None, 0, 1, x, x, x, x, x, x, x, stream=0),
                 lambda: qa.qa_q8_sparse_step_device_positions(None, 0, 1, x, 2, x, x, x, x, x, x, x, stream=0)):
        with pytest.raises(qa.QaError) as e:
            call()
        assert e.value.status == 1
    for bad in ([0.5], ["0"], 3, None, [None]):
        with pytest.raises(TypeError):
            qa.qa_q8_decode_step(None, 0, bad, x, x, x, x, x, x, stream=0)
    with pytest.raises(TypeError):
        qa.qa_q8_sparse_step(None, 0, [0], 0.5, x, x, x, x, x, x, x, stream=0)
    with pytest.raises(OverflowError):
        qa.qa_q8_sparse_step(None, 0, [0], 1 << 40, x, x, x, x, x, x, x, stream=0)
    with pytest.raises(ValueError):
        qa.qa_q8_append(None, 0, [0, 0], [1], 16, 16, stream=0)
    with pytest.raises(TypeError):
        qa._q4calls.q8_sparse(None, 0, [0], 1)
