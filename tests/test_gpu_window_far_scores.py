"""Windowed prefill when a row's visible scores lie far below zero (GPU).

A window can hide a block's first key tile from its later rows.  Their running
reference then starts at 0, and scores more than 2^-126 below it would all
vanish against it (0 / 0).  Here every row's visible scores are around -1000 in
units of log2: q is -k, so a token's score with itself is -|q'| |k'|.  The
expected values come from the definition in 64 bits on the kernels' own q' and
k' (tests/q4_ref.py); the tolerance is the prefill kernel's: one bf16 rounding
of the weights (2^-8, twice for the denominator) and one of the output, and an
error of a score of size |t| in fp32, 2^-24 |t| sqrt(D) < 2^-10 for |t| < 2^11."""
import pytest
import torch

import q4_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gqa_attention_preallocated_qa_gb300 import _build
    _build.build()
    from gqa_attention_preallocated_qa_gb300 import binding
    return binding


@pytest.mark.parametrize("hq,hkv,d,lens,window", [
    (8, 2, 128, [300], 2),             # one-CTA form
    (4, 4, 64, [300, 129], 3),
    (32, 8, 128, [700] * 4, 2),        # CTA pairs
])
@pytest.mark.parametrize("four_bits", [False, True])
def test_scores_far_below_zero_behind_a_hidden_tile(qa, hq, hkv, d, lens, window, four_bits):
    gen = torch.Generator(device="cuda").manual_seed(3)
    t, b, cap = sum(lens), len(lens), max(lens)
    k = torch.randn(t, hkv, d, generator=gen, device="cuda").bfloat16()
    v = torch.randn(t, hkv, d, generator=gen, device="cuda").bfloat16()
    q = (-k).repeat_interleave(hq // hkv, 1).contiguous()
    wq = torch.full((d,), 4.0, device="cuda").bfloat16()
    wk = torch.full((d,), 16.0 if d == 128 else 32.0, device="cuda").bfloat16()
    out, qp = torch.empty_like(q), torch.empty_like(q)
    h = qa.qa_cache_alloc(1, b, hq, hkv, d, cap)
    c4 = qa.qa_q4_cache_alloc(1, b, hq, hkv, d, cap)
    try:
        kt, vt, _ = qa.cache_tensors(h, 0, b, hkv, cap, d)
        qa.qa_prefill_transform(h, 0, lens, q, k, v, wq, wk, qp)
        if four_bits:
            qa.qa_q4_cache_set_window(c4, 0, window)
            qa.qa_q4_prefill(c4, 0, [0] * b, lens, q, k, v, wq, wk, out)
            kr, vr = torch.empty_like(k), torch.empty_like(v)
            qa.qa_q4_read(c4, 0, [0] * b, lens, kr, vr)
        else:
            kr = torch.cat([kt[i, :, :n].transpose(0, 1) for i, n in enumerate(lens)])
            vr = v
            qa.qa_cache_reset(h)
            qa.qa_cache_set_window(h, 0, window)
            qa.qa_prefill(h, 0, lens, q, k, v, wq, wk, out)
        at = 0
        for n in lens:
            s = slice(at, at + n)
            kk, vv = (x[s].double().transpose(0, 1) for x in (kr, vr))
            want, mag = q4_ref.attend(qp[s].double(), kk, vv, 0, window)
            tol = 2.0 ** -8 * want.abs() + (2.0 ** -7 + 2.0 ** -9) * mag + 1e-6
            assert ((out[s].double() - want).abs() <= tol).all()  # (false for NaN)
            at += n
    finally:
        qa.qa_cache_free(h)
        qa.qa_q4_cache_free(c4)
