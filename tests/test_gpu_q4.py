"""The 4-bit cache on the GPU against its definition in 64 bits (q4_ref.py).

Tolerances, from the roundings alone.  The values of a row are exact in bf16
and fp16, q' is exact in fp16, products and sums are fp32.  The decode kernel
rounds the weights P to fp16 (2^-11 relative), so an output moves by at most
2^-11 sum p|v| plus as much for the denominator, which uses the unrounded
weights: 2^-10 sum p|v|, with room for the fp32 sums and the 2-ulp exponential
(|t| < 2^6 here: 2^-17 relative); then one rounding to bf16, 2^-8 |out|.  The
prefill kernel rounds P to bf16: 2^-8 in the place of 2^-11, so 2^-7 sum p|v|.
"""
import numpy as np
import pytest
import torch

import q4_ref
from gpu_util import dev, f64

pytestmark = pytest.mark.gpu

THETA, EPS = 1e6, 1e-6


@pytest.fixture(scope="module")
def qa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gqa_attention_preallocated_qa_gb300 import _build
    _build.build()
    from gqa_attention_preallocated_qa_gb300 import binding
    return binding


def rows(seed, *shape, gain=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * gain).bfloat16()


class Cache:
    """A 4-bit cache beside a numpy copy of what it should hold."""

    def __init__(self, qa, layers, batch, hq, hkv, d, cap, seed=1):
        self.qa, self.hq, self.hkv, self.d, self.cap, self.batch = qa, hq, hkv, d, cap, batch
        self.h = qa.qa_q4_cache_alloc(layers, batch, hq, hkv, d, cap, THETA, EPS)
        self.bf16 = qa.qa_cache_alloc(1, batch, hq, hkv, d, cap, THETA, EPS)  # for its transform alone
        self.wq, self.wk = 1 + 0.1 * rows(seed, d), 1 + 0.1 * rows(seed + 1, d)
        rng = np.random.default_rng(seed)
        for layer in range(layers):  # poison: random codes under scales that are NaN or huge
            for i, t in enumerate(self.views(layer)):
                if i % 2:
                    t.copy_(torch.from_numpy(rng.choice([0x7F, 0x7C, 0x53], t.shape).astype(np.uint8)))
                else:
                    t.copy_(torch.from_numpy(rng.integers(0, 256, t.shape, dtype=np.uint8)))
        self.layer = [[x.cpu().numpy().copy() for x in self.views(l)] for l in range(layers)]

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.qa.qa_q4_cache_free(self.h)
        self.qa.qa_cache_free(self.bf16)

    def views(self, layer=0):
        return self.qa.q4_cache_tensors(self.h, layer, self.batch, self.hkv, self.cap, self.d)

    def note(self, layer, start, ntok, k, v):
        """k, v float64 [T, Hkv, D] (transformed) into the copy; the rows' values."""
        held = []
        for i, x in ((0, k), (2, v)):
            codes, scales = q4_ref.quantise(x)
            at = 0
            for b, (s, n) in enumerate(zip(start, ntok)):
                self.layer[layer][i][b, :, s:s + n] = codes[at:at + n].swapaxes(0, 1)
                self.layer[layer][i + 1][b, :, s:s + n] = scales[at:at + n].swapaxes(0, 1)
                at += n
            held.append(q4_ref.values(codes, scales))
        return held

    def check_bytes(self, layer=0):
        for got, want in zip(self.views(layer), self.layer[layer]):
            np.testing.assert_array_equal(got.cpu().numpy(), want)

    def transform(self, start, ntok, q, k, v):
        """q', k' of the bf16 path (K1), which the 4-bit path shares, as float64."""
        kt, _, _ = self.qa.cache_tensors(self.bf16, 0, self.batch, self.hkv, self.cap, self.d)
        self.qa.qa_cache_set_lengths(self.bf16, 0, list(start) + [0] * (self.batch - len(start)))
        qp = torch.empty_like(q)
        self.qa.qa_prefill_transform(self.bf16, 0, list(ntok), q, k, v, self.wq, self.wk, qp)
        kp = torch.cat([kt[b, :, s:s + n].transpose(0, 1) for b, (s, n) in enumerate(zip(start, ntok))])
        return qp.double(), kp.double().cpu().numpy()

    def want(self, start, ntok, qp, layer=0, window=0):
        outs, mags, at = [], [], 0
        for b, (s, n) in enumerate(zip(start, ntok)):
            if n == 0:
                continue
            kc, ks, vc, vs = (x[b, :, :s + n] for x in self.layer[layer])
            kk, vv = (torch.from_numpy(q4_ref.values(c, x)).cuda() for c, x in ((kc, ks), (vc, vs)))
            lo = max(0, s + 1 - window) if window else 0  # rows below are seen by none
            o, m = q4_ref.attend(qp[at:at + n], kk[:, lo:], vv[:, lo:], s - lo, window)
            outs.append(o)
            mags.append(m)
            at += n
        return torch.cat(outs), torch.cat(mags)

    def fill(self, layer, lens, seed):
        """Rows 0..lens[b] - 1 of each sequence through append."""
        k, v = rows(seed, sum(lens), self.hkv, self.d), rows(seed + 1, sum(lens), self.hkv, self.d)
        zero = [0] * len(lens)
        self.qa.qa_q4_append(self.h, layer, zero, lens, k, v)
        self.note(layer, zero, lens, f64(k), f64(v))

    def tokens(self, ntok, seed):
        t = sum(ntok)
        return rows(seed, t, self.hq, self.d), rows(seed + 1, t, self.hkv, self.d), rows(seed + 2, t, self.hkv, self.d)


def close(got, want, mag, p_bits, what=""):
    got = got.double()
    tol = 2.0 ** -8 * want.abs() + 2.0 ** (1 - p_bits) * mag + 1e-6
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {float(((got - want).abs() / tol).max()):.3f} of the tolerance"


DECODE_BITS, PREFILL_BITS = 11, 8


# ------------------------------------------------------------------ rows
@pytest.mark.parametrize("d", [64, 128])
def test_append_is_the_definition(qa, d):
    # Every bf16 magnitude as a group's largest, with values that hit halves of
    # the steps of its scale; groups of zeros, of subnormals, past the largest scale.
    rng = np.random.default_rng(d)
    bits = rng.permutation(np.arange(0, 0x7E80, 3)).astype(np.uint32)
    n = bits.size // (d // 32)
    x = np.zeros((n, 4, d), np.float32)
    g = x.reshape(-1, 32)
    top = (bits << 16).view(np.float32)[np.arange(g.shape[0]) % bits.size]
    g[:] = rng.uniform(-1, 1, g.shape).astype(np.float32) * top[:, None]
    halves = rng.integers(-15, 16, g.shape) / np.float32(14)
    pick = rng.random(g.shape) < 0.5
    g[pick] = (halves * top[:, None])[pick]
    g[np.arange(g.shape[0]), rng.integers(0, 32, g.shape[0])] = top * rng.choice([-1, 1], g.shape[0])
    k = torch.from_numpy(x).cuda().bfloat16()
    v = k.flip(0).contiguous()
    with Cache(qa, 1, 1, 8, 4, d, n) as c:
        kh, vh = torch.empty_like(k), torch.empty_like(v)
        qa.qa_q4_append(c.h, 0, [0], [n], k, v, kh, vh)
        held = c.note(0, [0], [n], f64(k), f64(v))
        c.check_bytes()
        np.testing.assert_array_equal(f64(kh), held[0])
        np.testing.assert_array_equal(f64(vh), held[1])
        kr, vr = torch.empty_like(k), torch.empty_like(v)
        qa.qa_q4_read(c.h, 0, [0], [n], kr, vr)
        assert torch.equal(kr, kh) and torch.equal(vr, vh)


@pytest.mark.parametrize("d,hkv", [(64, 1), (128, 8), (128, 3)])
def test_append_and_read_ranges(qa, d, hkv):
    start, ntok = [0, 17, 5, 99, 0], [33, 1, 0, 16, 64]
    with Cache(qa, 2, 5, hkv, hkv, d, 130) as c:
        _, k, v = c.tokens(ntok, 7)
        kh, vh = k.clone(), v.clone()
        qa.qa_q4_append(c.h, 1, start, ntok, kh, vh, kh, vh)  # the values in place of the rows
        held = c.note(1, start, ntok, f64(k), f64(v))
        for layer in (0, 1):
            c.check_bytes(layer)
        np.testing.assert_array_equal(f64(kh), held[0])
        np.testing.assert_array_equal(f64(vh), held[1])
        out = torch.full_like(k, 7.0)
        qa.qa_q4_read(c.h, 1, start, ntok, None, out)
        np.testing.assert_array_equal(f64(out), held[1])
        qa.qa_q4_read(c.h, 1, start, ntok, out, None)
        np.testing.assert_array_equal(f64(out), held[0])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_groups_with_values_that_are_not_finite(qa, bad):
    with Cache(qa, 1, 1, 2, 2, 128, 40) as c:
        _, k, v = c.tokens([40], 3)
        k[3, 1, 5] = bad
        v[39, 0, 127] = bad
        kh, vh = torch.empty_like(k), torch.empty_like(v)
        qa.qa_q4_append(c.h, 0, [0], [40], k, v, kh, vh)
        c.note(0, [0], [40], f64(k), f64(v))
        c.check_bytes()
        for x, (t, h, g) in ((kh, (3, 1, 0)), (vh, (39, 0, 3))):
            nan = torch.isnan(x)
            assert nan[t, h, 32 * g:32 * g + 32].all() and int(nan.sum()) == 32


# ------------------------------------------------------------------ decode
SHAPES = [(32, 8, 128), (8, 8, 64), (8, 1, 128), (4, 2, 64), (8, 1, 64), (3, 3, 128), (6, 3, 128)]


@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("lens", [[0], [1], [31, 32, 33], [64, 255, 0, 257], [1500, 7]])
def test_decode_step(qa, hq, hkv, d, lens):
    one = [1] * len(lens)
    with Cache(qa, 2, len(lens), hq, hkv, d, max(lens) + 1) as c:
        c.fill(1, lens, 11)
        q, k, v = c.tokens(one, 21)
        out, kh, vh = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        qa.qa_q4_decode_step(c.h, 1, lens, q, k, v, c.wq, c.wk, out, kh, vh)
        qp, kp = c.transform(lens, one, q, k, v)
        held = c.note(1, lens, one, kp, f64(v))
        assert qa.qa_q4_get_device_error(c.h) == (0, 0)
        c.check_bytes(0)
        c.check_bytes(1)
        np.testing.assert_array_equal(f64(kh), held[0])
        np.testing.assert_array_equal(f64(vh), held[1])
        want, mag = c.want(lens, one, qp, 1)
        close(out, want, mag, DECODE_BITS)


def test_decode_long_cache_and_peaked_scores(qa):
    # 40,000 keys; queries scaled so that a few keys carry a row.
    lens = [40000, 39001]
    with Cache(qa, 1, 2, 8, 2, 128, 40001) as c:
        c.fill(0, lens, 5)
        c.wq = c.wq * 4
        q, k, v = c.tokens([1, 1], 6)
        out = torch.empty_like(q)
        qa.qa_q4_decode_step(c.h, 0, lens, q, k, v, c.wq, c.wk, out)
        qp, kp = c.transform(lens, [1, 1], q, k, v)
        c.note(0, lens, [1, 1], kp, f64(v))
        want, mag = c.want(lens, [1, 1], qp)
        close(out, want, mag, DECODE_BITS)


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (4, 2, 64), (8, 1, 64), (3, 3, 128), (6, 3, 128)])
@pytest.mark.parametrize("tokens", [1, 3])
@pytest.mark.parametrize("lens", [[300, 90, 9000, 7], [100, 6000, 33, 2500, 0, 1200, 700, 300, 7], [5000] + [17] * 12])
def test_decode_batches_of_mixed_lengths(qa, hq, hkv, d, tokens, lens):
    # Lengths that get different numbers of splits: several groups in a cluster,
    # the last cluster filled up (3 kv heads).
    ntok = [tokens] * len(lens)
    with Cache(qa, 1, len(lens), hq, hkv, d, max(lens) + 8) as c:
        c.fill(0, lens, 5)
        q, k, v = c.tokens(ntok, 6)
        outs = [torch.full_like(q, float("nan")) for _ in range(2)]
        for out in outs:
            if tokens == 1:
                qa.qa_q4_decode_step(c.h, 0, lens, q, k, v, c.wq, c.wk, out)
            else:
                qa.qa_q4_prefill(c.h, 0, lens, ntok, q, k, v, c.wq, c.wk, out)
        assert qa.qa_q4_get_device_error(c.h) == (0, 0)
        assert torch.equal(*outs)
        qp, kp = c.transform(lens, ntok, q, k, v)
        c.note(0, lens, ntok, kp, f64(v))
        c.check_bytes()
        want, mag = c.want(lens, ntok, qp)
        close(outs[0], want, mag, DECODE_BITS)


def test_decode_more_sequences_than_a_launch(qa):
    lens = [(i * 37) % 150 for i in range(70)]
    one = [1] * 70
    with Cache(qa, 1, 70, 4, 1, 128, 160) as c:
        c.fill(0, lens, 5)
        q, k, v = c.tokens(one, 6)
        out = torch.empty_like(q)
        qa.qa_q4_decode_step(c.h, 0, lens, q, k, v, c.wq, c.wk, out)
        qp, kp = c.transform(lens, one, q, k, v)
        c.note(0, lens, one, kp, f64(v))
        c.check_bytes()
        want, mag = c.want(lens, one, qp)
        close(out, want, mag, DECODE_BITS)
        assert qa.qa_q4_stats(c.h)["decode"] == 2


@pytest.mark.parametrize("window", [1, 2, 33, 100, 5000])
def test_decode_window(qa, window):
    lens = [0, 99, 100, 301]
    one = [1] * 4
    with Cache(qa, 1, 4, 8, 2, 128, 302) as c:
        qa.qa_q4_cache_set_window(c.h, 0, window)
        c.fill(0, lens, 5)
        for b, n in enumerate(lens):  # rows below the window may hold anything
            below = max(0, n + 1 - window)
            for i in (1, 3):
                c.views()[i][b, :, :below] = 0x7F
                c.layer[0][i][b, :, :below] = 0x7F
        q, k, v = c.tokens(one, 6)
        out = torch.empty_like(q)
        qa.qa_q4_decode_step(c.h, 0, lens, q, k, v, c.wq, c.wk, out)
        qp, kp = c.transform(lens, one, q, k, v)
        c.note(0, lens, one, kp, f64(v))
        want, mag = c.want(lens, one, qp, window=window)
        close(out, want, mag, DECODE_BITS)


def test_decode_nan_key_reaches_the_heads_that_see_it(qa):
    lens, one = [40, 40], [1, 1]
    with Cache(qa, 1, 2, 4, 2, 128, 64) as c:
        c.fill(0, lens, 5)
        c.views()[1][1, 0, 20, 2] = 0x7F  # a group of a key of sequence 1, kv head 0
        q, k, v = c.tokens(one, 6)
        out = torch.empty_like(q)
        qa.qa_q4_decode_step(c.h, 0, lens, q, k, v, c.wq, c.wk, out)
        nan = torch.isnan(out).all(-1)
        assert nan.tolist() == [[False] * 4, [True, True, False, False]]


def test_decode_is_the_same_every_time(qa):
    lens, one = [2000, 1111, 3], [1] * 3
    with Cache(qa, 1, 3, 32, 8, 128, 2001) as c:
        c.fill(0, lens, 5)
        q, k, v = c.tokens(one, 6)
        outs = []
        for _ in range(5):
            out = torch.empty_like(q)
            qa.qa_q4_decode_step(c.h, 0, lens, q, k, v, c.wq, c.wk, out)
            outs.append(out)
        assert all(torch.equal(o, outs[0]) for o in outs)


# ------------------------------------------------------------------ several tokens
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 1, 64), (4, 4, 64), (4, 2, 128)])
@pytest.mark.parametrize("window", [0, 3, 40])
def test_short_chunk(qa, hq, hkv, d, window):
    start, ntok = [0, 65, 33, 500, 7], [8, 2, 0, 5, 1]
    with Cache(qa, 1, 5, hq, hkv, d, 520) as c:
        qa.qa_q4_cache_set_window(c.h, 0, window)
        c.fill(0, start, 5)
        q, k, v = c.tokens(ntok, 6)
        out = torch.empty_like(q)
        qa.qa_q4_prefill(c.h, 0, start, ntok, q, k, v, c.wq, c.wk, out)
        qp, kp = c.transform(start, ntok, q, k, v)
        c.note(0, start, ntok, kp, f64(v))
        c.check_bytes()
        want, mag = c.want(start, ntok, qp, window=window)
        close(out, want, mag, DECODE_BITS)
        assert qa.qa_q4_stats(c.h)["decode"] == 1 and qa.qa_q4_stats(c.h)["prefill_attn"] == 0


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 1, 64), (3, 3, 128)])
@pytest.mark.parametrize("window", [0, 600])
def test_chunks_of_several_launches_beside_long_ones(qa, hq, hkv, d, window):
    # Each sequence by its own length: up to 16, 24 or 32 tokens in the decode
    # kernel, eight at a time; the longer ones, in groups with those between them
    # left out, in the prefill kernel.
    start, ntok = [100, 0, 6000, 0, 0, 700, 33, 511, 5, 4100], [1, 300, 24, 16, 0, 24, 17, 16, 40, 9]
    long = [17 <= n and (n > 24 or s < 512) for s, n in zip(start, ntok)]
    with Cache(qa, 1, len(start), hq, hkv, d, 6040) as c:
        qa.qa_q4_cache_set_window(c.h, 0, window)
        c.fill(0, start, 5)
        q, k, v = c.tokens(ntok, 6)
        out = torch.full_like(q, float("nan"))
        qa.qa_q4_prefill(c.h, 0, start, ntok, q, k, v, c.wq, c.wk, out)
        assert qa.qa_q4_get_device_error(c.h) == (0, 0)
        assert qa.qa_q4_stats(c.h)["decode"] == 3 and qa.qa_q4_stats(c.h)["prefill_attn"] == 3
        qp, kp = c.transform(start, ntok, q, k, v)
        c.note(0, start, ntok, kp, f64(v))
        c.check_bytes()
        want, mag = c.want(start, ntok, qp, window=window)
        rows = torch.tensor(long).repeat_interleave(torch.tensor(ntok)).cuda()
        close(out[rows], want[rows], mag[rows], PREFILL_BITS)
        close(out[~rows], want[~rows], mag[~rows], DECODE_BITS)


def test_chunk_of_sixteen_in_a_graph(qa):
    # The same chunk replayed: written twice, the same bits as the eager call.
    start, ntok = [40, 300], [16, 13]
    with Cache(qa, 1, 2, 8, 2, 128, 330) as c:
        c.fill(0, start, 5)
        q, k, v = c.tokens(ntok, 6)
        eager, out = torch.empty_like(q), torch.empty_like(q)
        qa.qa_q4_prefill(c.h, 0, start, ntok, q, k, v, c.wq, c.wk, eager)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            qa.qa_q4_prefill(c.h, 0, start, ntok, q, k, v, c.wq, c.wk, out)
        qp, kp = c.transform(start, ntok, q, k, v)
        c.note(0, start, ntok, kp, f64(v))
        want, mag = c.want(start, ntok, qp)
        for _ in range(2):
            out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, eager)
        close(out, want, mag, DECODE_BITS)
        c.check_bytes()


# ------------------------------------------------------------------ prefill
@pytest.mark.parametrize("hq,hkv,d,start,ntok,window", [
    (8, 2, 128, [0], [9], 0),
    (2, 1, 64, [0], [64], 0),
    (8, 2, 128, [0, 0, 0], [129, 1, 300], 0),
    (4, 4, 64, [100, 0, 257], [130, 40, 255], 0),
    (8, 1, 128, [300, 140], [200, 77], 150),
    (32, 8, 128, [1500, 130, 20, 1500], [700, 900, 60, 130], 0),  # more blocks than the device takes at once
    (16, 8, 64, [900, 0], [300, 1000], 700),
    (32, 8, 128, [2000, 1500, 1800, 2000, 700], [100, 90, 128, 33, 64], 0),  # two-head items, fewer than SMs
    (16, 8, 64, [900] * 6, [200] * 6, 300),
    (4, 1, 64, [31] * 11, [20, 0, 3, 150, 9, 1, 20, 33, 128, 2, 17], 0),
])
def test_prefill(qa, hq, hkv, d, start, ntok, window):
    cap = max(s + n for s, n in zip(start, ntok))
    with Cache(qa, 1, len(start), hq, hkv, d, cap) as c:
        qa.qa_q4_cache_set_window(c.h, 0, window)
        c.fill(0, start, 5)
        q, k, v = c.tokens(ntok, 6)
        out = torch.full_like(q, float("nan"))
        qa.qa_q4_prefill(c.h, 0, start, ntok, q, k, v, c.wq, c.wk, out)
        qp, kp = c.transform(start, ntok, q, k, v)
        c.note(0, start, ntok, kp, f64(v))
        c.check_bytes()
        want, mag = c.want(start, ntok, qp, window=window)
        close(out, want, mag, PREFILL_BITS)
        assert qa.qa_q4_get_device_error(c.h) == (0, 0)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("hq,hkv,d,start,ntok,window", [
    (8, 2, 128, [5000], [100], 0),
    (32, 8, 128, [6001, 2500], [60, 33], 0),
    (8, 1, 64, [9000], [300], 0),
    (4, 4, 64, [5000, 0, 300], [130, 40, 257], 0),     # one sequence with parts, others without
    (3, 3, 128, [4096], [128], 0),
    (8, 2, 128, [9000], [257], 3000),                   # the window starts inside the first part
    (16, 8, 64, [7000, 40], [129, 33], 2500),
    (4, 2, 128, [8191], [40], 8000),
])
def test_prefill_keys_in_parts(qa, hq, hkv, d, start, ntok, window):
    # Few query blocks behind many keys: the keys are cut into parts and joined.
    with Cache(qa, 1, len(start), hq, hkv, d, max(start) + max(ntok)) as c:
        qa.qa_q4_cache_set_window(c.h, 0, window)
        c.fill(0, start, 5)
        q, k, v = c.tokens(ntok, 6)
        outs = [torch.full_like(q, float("nan")) for _ in range(2)]
        for out in outs:
            qa.qa_q4_prefill(c.h, 0, start, ntok, q, k, v, c.wq, c.wk, out)
        assert qa.qa_q4_get_device_error(c.h) == (0, 0)
        assert torch.equal(*outs)
        qp, kp = c.transform(start, ntok, q, k, v)
        c.note(0, start, ntok, kp, f64(v))
        c.check_bytes()
        want, mag = c.want(start, ntok, qp, window=window)
        close(outs[0], want, mag, PREFILL_BITS)


def test_generate_steps_back_to_back(qa):
    # A prompt, then decode steps over two layers with nothing between the
    # launches, a verify chunk whose last tokens are dropped, and more steps.
    layers, prompt = 2, [130, 70]
    with Cache(qa, layers, 2, 8, 2, 128, 256) as c:
        plan = [(list(prompt), True)] + [([1, 1], False)] * 9 + [([4, 4], True)] + [([1, 1], False)] * 6
        pos, calls = [0, 0], []
        for i, (ntok, chunk) in enumerate(plan):
            if i == 11:
                pos = [p - 3 for p in pos]  # one of four verified tokens was kept
            for layer in range(layers):
                q, k, v = c.tokens(ntok, 100 * i + 10 * layer)
                calls.append((layer, list(pos), ntok, chunk, q, k, v, torch.empty_like(q)))
            pos = [p + n for p, n in zip(pos, ntok)]
        torch.cuda.synchronize()
        for layer, start, ntok, chunk, q, k, v, out in calls:
            if chunk:
                qa.qa_q4_prefill(c.h, layer, start, ntok, q, k, v, c.wq, c.wk, out)
            else:
                qa.qa_q4_decode_step(c.h, layer, start, q, k, v, c.wq, c.wk, out)
        torch.cuda.synchronize()
        for layer, start, ntok, chunk, q, k, v, out in calls:
            qp, kp = c.transform(start, ntok, q, k, v)
            c.note(layer, start, ntok, kp, f64(v))
            want, mag = c.want(start, ntok, qp, layer)
            close(out, want, mag, PREFILL_BITS if ntok[0] > 8 else DECODE_BITS, f"at {start}")
        for layer in range(layers):
            c.check_bytes(layer)


def test_prefill_then_chunks_equal_one_read_back(qa):
    # Rows written as one prompt, as chunks and one by one are the same bytes.
    n, steps = 96, [40, 8, 30, 1, 1, 16]
    with Cache(qa, 2, 1, 8, 2, 128, n) as c:
        q, k, v = c.tokens([n], 6)
        out = torch.empty_like(q)
        qa.qa_q4_prefill(c.h, 0, [0], [n], q, k, v, c.wq, c.wk, out)
        at = 0
        for m in steps:
            sl = slice(at, at + m)
            o = torch.empty_like(q[sl])
            qa.qa_q4_prefill(c.h, 1, [at], [m], q[sl], k[sl], v[sl], c.wq, c.wk, o)
            at += m
        assert at == n
        for a, b in zip(c.views(0), c.views(1)):
            assert torch.equal(a, b)


def test_device_positions_in_a_graph(qa):
    lens, one = [60, 95], [1, 1]
    with Cache(qa, 1, 2, 8, 2, 128, 128) as c:
        c.fill(0, lens, 5)
        q, k, v = c.tokens(one, 6)
        pos = torch.tensor(lens, dtype=torch.int32, device="cuda")
        out = torch.empty_like(q)

        def step():
            qa.qa_q4_decode_step_device_positions(c.h, 0, 2, pos, q, k, v, c.wq, c.wk, out)
            pos.add_(1)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for i in range(6):
            at = [x + i for x in lens]
            if i:
                fresh = c.tokens(one, 50 + i)
                for a, b in zip((q, k, v), fresh):
                    a.copy_(b)
                graph.replay()
            torch.cuda.synchronize()
            qp, kp = c.transform(at, one, q, k, v)
            c.note(0, at, one, kp, f64(v))
            want, mag = c.want(at, one, qp)
            close(out, want, mag, DECODE_BITS, f"step {i}")
        c.check_bytes()
        assert pos.tolist() == [x + 6 for x in lens]


def test_device_position_out_of_range_is_reported(qa):
    with Cache(qa, 1, 3, 8, 2, 128, 64) as c:
        lens = [10, 20, 30]
        c.fill(0, lens, 5)
        q, k, v = c.tokens([1] * 3, 6)
        out = torch.full_like(q, 5.0)
        pos = torch.tensor([10, 64, -1], dtype=torch.int32, device="cuda")
        qa.qa_q4_decode_step_device_positions(c.h, 0, 3, pos, q, k, v, c.wq, c.wk, out)
        st, _ = qa.qa_q4_get_device_error(c.h)
        assert st == 8
        assert (out[1:] == 5.0).all() and (out[0] != 5.0).any()
        qp, kp = c.transform([10], [1], q[:1], k[:1], v[:1])
        c.note(0, [10], [1], kp, f64(v[:1]))
        c.check_bytes()


def test_prefill_on_two_streams_shares_the_workspace(qa):
    ntok = [200, 150]
    with Cache(qa, 2, 2, 8, 2, 128, 200) as c:
        sets = [(l, *c.tokens(ntok, 30 + l)) for l in (0, 1)]
        outs = [torch.empty_like(s[1]) for s in sets]
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for _ in range(4):
            for (l, q, k, v), out, st in zip(sets, outs, streams):
                qa.qa_q4_prefill(c.h, l, [0, 0], ntok, q, k, v, c.wq, c.wk, out, stream=st)
        torch.cuda.synchronize()
        for (l, q, k, v), out in zip(sets, outs):
            qp, kp = c.transform([0, 0], ntok, q, k, v)
            c.note(l, [0, 0], ntok, kp, f64(v))
            want, mag = c.want([0, 0], ntok, qp, l)
            close(out, want, mag, PREFILL_BITS)


# ------------------------------------------------------------------ refusals
def test_refusals_change_nothing(qa):
    with Cache(qa, 1, 2, 8, 2, 128, 64) as c:
        c.fill(0, [20, 20], 5)
        q, k, v = c.tokens([17, 9], 6)
        out = torch.full_like(q, 3.0)
        w = (c.wq, c.wk)

        def refused(status, fn, *args):
            with pytest.raises(qa.QaError) as e:
                fn(c.h, *args)
            assert e.value.status == status, args

        odd = q.view(-1)[1:]
        for layer in (-1, 1):
            refused(1, qa.qa_q4_append, layer, [0], [1], k, v)
            refused(1, qa.qa_q4_decode_step, layer, [0], q, k, v, *w, out)
        refused(1, qa.qa_q4_append, 0, [0, 0, 0], [1, 1, 1], k, v)      # more than max_batch
        refused(1, qa.qa_q4_append, 0, [], [], k, v)
        refused(1, qa.qa_q4_append, 0, [-1], [1], k, v)
        refused(1, qa.qa_q4_append, 0, [0], [-1], k, v)
        refused(4, qa.qa_q4_append, 0, [60, 0], [5, 1], k, v)
        refused(4, qa.qa_q4_append, 0, [2 ** 31 - 1], [2 ** 31 - 1], k, v)
        refused(1, qa.qa_q4_append, 0, [0], [1], None, v)
        refused(1, qa.qa_q4_append, 0, [0], [1], k, v, k, None)
        refused(3, qa.qa_q4_append, 0, [0], [1], odd, v)
        refused(4, qa.qa_q4_read, 0, [64], [1], k, v)
        refused(1, qa.qa_q4_read, 0, [0], [1], None, None)
        refused(3, qa.qa_q4_read, 0, [0], [1], k, odd)
        for n in (3, 9, 17):
            refused(4, qa.qa_q4_prefill, 0, [60], [n + 2], q, k, v, *w, out)
            refused(1, qa.qa_q4_prefill, 0, [0], [n], q, k, v, None, c.wk, out)
            refused(3, qa.qa_q4_prefill, 0, [0], [n], q, k, v, *w, odd)
        refused(4, qa.qa_q4_decode_step, 0, [64, 0], q, k, v, *w, out)
        refused(1, qa.qa_q4_decode_step, 0, [0, -1], q, k, v, *w, out)
        refused(1, qa.qa_q4_decode_step, 0, [0], q, k, v, *w, None)
        refused(1, qa.qa_q4_decode_step, 0, [0], q, k, v, *w, out, k, None)
        refused(3, qa.qa_q4_decode_step, 0, [0], q, odd, v, *w, out)
        refused(1, qa.qa_q4_decode_step_device_positions, 0, 1, None, q, k, v, *w, out)
        refused(1, qa.qa_q4_cache_set_window, 0, -1)
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.stream(side):
            graph.capture_begin()
            try:
                refused(5, qa.qa_q4_prefill, 0, [20], [17], q, k, v, *w, out, side)
            finally:
                graph.capture_end()
        torch.cuda.synchronize()
        assert (out == 3.0).all()
        c.check_bytes()
        qa.qa_q4_append(c.h, 0, [0, 64], [0, 0], None, None)  # no rows: nothing to do
        assert qa.qa_q4_stats(c.h) == {"norm_rope": 0, "quantise": 1, "dequantise": 0, "prefill_attn": 0, "decode": 0}


def test_memory_info(qa):
    c = qa.qa_q4_cache_alloc(3, 10, 8, 2, 128, 100)
    try:
        held, scratch = qa.qa_q4_memory_info(c)
        assert held == 2 * 3 * 10 * 2 * 128 * (64 + 4)
        assert scratch >= 2 * 8 * 2 * 100 * 128 * 2
    finally:
        qa.qa_q4_cache_free(c)


def test_sequences_behind_the_batch_are_left_alone(qa):
    # A cache of four sequences, calls on the first two: the others' bytes stay.
    with Cache(qa, 1, 4, 8, 2, 128, 160) as c:
        c.fill(0, [64, 100], 5)
        for ntok, what in (([1, 1], "step"), ([3, 2], "chunk"), ([20, 9], "prefill")):
            start = [64, 100] if what == "step" else [65, 101] if what == "chunk" else [68, 103]
            q, k, v = c.tokens(ntok, 6)
            out = torch.empty_like(q)
            if what == "step":
                qa.qa_q4_decode_step(c.h, 0, start, q, k, v, c.wq, c.wk, out)
            else:
                qa.qa_q4_prefill(c.h, 0, start, ntok, q, k, v, c.wq, c.wk, out)
            qp, kp = c.transform(start, ntok, q, k, v)
            c.note(0, start, ntok, kp, f64(v))
            c.check_bytes()
            want, mag = c.want(start, ntok, qp)
            close(out, want, mag, PREFILL_BITS if max(ntok) > 8 else DECODE_BITS, what)


def test_offsets_past_32_bits(qa):
    # 2^26 rows of K and of V: 2^32 bytes of codes each; the last sequence lies
    # behind that border, and its last rows at its end.
    cap, batch, hkv = 1 << 19, 16, 8
    h = qa.qa_q4_cache_alloc(1, batch, hkv, hkv, 128, cap, THETA, EPS)
    try:
        n = 300
        start, ntok = [0] * 15 + [cap - n - 1], [1] * 15 + [n]
        k, v = rows(1, sum(ntok), hkv, 128), rows(2, sum(ntok), hkv, 128)
        kh, vh = torch.empty_like(k), torch.empty_like(v)
        qa.qa_q4_append(h, 0, start, ntok, k, v, kh, vh)
        kr, vr = torch.empty_like(k), torch.empty_like(v)
        qa.qa_q4_read(h, 0, start, ntok, kr, vr)
        assert torch.equal(kr, kh) and torch.equal(vr, vh)
        codes, scales = q4_ref.quantise(f64(k))
        np.testing.assert_array_equal(f64(kh), q4_ref.values(codes, scales))
        # A window keeps the step on the rows that were written.
        qa.qa_q4_cache_set_window(h, 0, n + 1)
        one = torch.ones(128, device="cuda").bfloat16()
        pos = [1] * 15 + [cap - 1]
        q, kn, vn = rows(3, 16, hkv, 128), rows(4, 16, hkv, 128), rows(5, 16, hkv, 128)
        out, kn_h, vn_h = torch.empty_like(q), torch.empty_like(kn), torch.empty_like(vn)
        qa.qa_q4_decode_step(h, 0, pos, q, kn, vn, one, one, out, kn_h, vn_h)
        assert qa.qa_q4_get_device_error(h) == (0, 0)
        # the last sequence's step, against its rows as they are held
        ang = (cap - 1) * THETA ** (-2.0 * np.arange(64) / 128)
        f = q[15].double()
        y = (f / torch.sqrt((f * f).mean(-1, keepdim=True) + EPS)).bfloat16().double()
        cs, sn = torch.from_numpy(np.cos(ang)).cuda(), torch.from_numpy(np.sin(ang)).cuda()
        qp = torch.cat((y[:, :64] * cs - y[:, 64:] * sn, y[:, 64:] * cs + y[:, :64] * sn), -1).bfloat16().double()
        kk = torch.cat((kh[15:].double(), kn_h[15:].double())).transpose(0, 1)
        vv = torch.cat((vh[15:].double(), vn_h[15:].double())).transpose(0, 1)
        want, mag = q4_ref.attend(qp[None], kk, vv, n)
        # A query rounded the other way by the kernel's fp32 root moves a score by
        # 2^-8 |q_i k_i| / sqrt(D): below 2^-8 * 4 * 4 / 11 = 2^-8 * 1.5 of a weight's size.
        close(out[15:], want, mag, 7)
    finally:
        qa.qa_q4_cache_free(h)


def test_steps_beside_a_bf16_cache_on_one_stream(qa):
    # Both caches' decode steps back to back, as a model with some layers in each
    # would make them: neither disturbs the other's order.
    steps = 12
    with Cache(qa, 1, 2, 8, 2, 128, 128) as c:
        c.fill(0, [100, 37], 5)
        h = qa.qa_cache_alloc(1, 2, 8, 2, 128, 128, THETA, EPS)
        try:
            ks, vs, _ = qa.cache_tensors(h, 0, 2, 2, 128, 128)
            ks.copy_(rows(71, 2, 2, 128, 128))
            vs.copy_(rows(72, 2, 2, 128, 128))
            qa.qa_cache_set_lengths(h, 0, [100, 37])
            calls = [(c.tokens([1, 1], 300 + 10 * i), [100 + i, 37 + i]) for i in range(steps)]
            got4, got16 = ([torch.empty_like(x[0][0]) for x in calls] for _ in range(2))
            torch.cuda.synchronize()
            for ((q, k, v), pos), o4, o16 in zip(calls, got4, got16):
                qa.qa_q4_decode_step(c.h, 0, pos, q, k, v, c.wq, c.wk, o4)
                qa.qa_decode_step(h, 0, 2, q, k, v, c.wq, c.wk, o16)
            torch.cuda.synchronize()
            for i, ((q, k, v), pos) in enumerate(calls):
                qp, kp = c.transform(pos, [1, 1], q, k, v)
                c.note(0, pos, [1, 1], kp, f64(v))
                want, mag = c.want(pos, [1, 1], qp)
                close(got4[i], want, mag, DECODE_BITS, f"4-bit step {i}")
                kp = torch.from_numpy(kp).cuda()
                outs = [q4_ref.attend(qp[b:b + 1],
                                      torch.cat((ks[b, :, :n].double(), kp[b, :, None]), 1),
                                      torch.cat((vs[b, :, :n].double(), v[b, :, None].double()), 1), n) for b, n in enumerate(pos)]
                close(got16[i], torch.cat([o for o, _ in outs]), torch.cat([m for _, m in outs]), PREFILL_BITS, f"bf16 step {i}")
        finally:
            qa.qa_cache_free(h)


def test_calls_allocate_nothing(qa):
    with Cache(qa, 1, 2, 8, 2, 128, 600) as c:
        sets = {n: c.tokens([n, n], n) for n in (1, 4, 200)}
        outs = {n: torch.empty_like(s[0]) for n, s in sets.items()}

        def calls():
            for n, (q, k, v) in sets.items():
                qa.qa_q4_prefill(c.h, 0, [300, 7], [n, n], q, k, v, c.wq, c.wk, outs[n])
                qa.qa_q4_append(c.h, 0, [300, 7], [n, n], k, v)
                qa.qa_q4_read(c.h, 0, [300, 7], [n, n], k, v)
            qa.qa_q4_decode_step(c.h, 0, [300, 7], *sets[1], c.wq, c.wk, outs[1])
            torch.cuda.synchronize()

        calls()
        free = torch.cuda.mem_get_info()[0]
        for _ in range(20):
            calls()
        assert torch.cuda.mem_get_info()[0] == free


def test_a_wait_that_runs_out_is_reported_and_the_cache_stays_usable(qa):
    lens = [700, 300]
    with Cache(qa, 1, 2, 32, 8, 128, 1024) as c:
        c.fill(0, lens, 5)
        q, k, v = c.tokens([1, 1], 6)
        out = torch.empty_like(q)
        qa.qa_debug_arm_wait_timeout(2, 20000)  # the next decode launch: 20 ms
        qa.qa_q4_decode_step(c.h, 0, lens, q, k, v, c.wq, c.wk, out)
        st, word = qa.qa_q4_get_device_error(c.h)
        assert st == 7 and word & 0xff == 1 and word >> 8 & 0xff == 5
        assert qa.qa_q4_get_device_error(c.h) == (0, 0)
        qa.qa_q4_decode_step(c.h, 0, lens, q, k, v, c.wq, c.wk, out)
        assert qa.qa_q4_get_device_error(c.h) == (0, 0)
        qp, kp = c.transform(lens, [1, 1], q, k, v)
        c.note(0, lens, [1, 1], kp, f64(v))
        want, mag = c.want(lens, [1, 1], qp)
        close(out, want, mag, DECODE_BITS)


@pytest.mark.parametrize("lens,ntok,kernel", [
    ([300, 4000, 90, 7], [1] * 4, 2),       # splits by length, several groups in a cluster
    ([5000, 0], [100, 0], 1),               # the prefill kernel with the keys in parts, and the join behind it
])
def test_a_wait_that_runs_out_in_the_other_forms(qa, lens, ntok, kernel):
    with Cache(qa, 1, len(lens), 32, 8, 128, 5200) as c:
        c.fill(0, lens, 5)
        q, k, v = c.tokens(ntok, 6)
        out = torch.empty_like(q)
        qa.qa_debug_arm_wait_timeout(kernel, 20000)
        qa.qa_q4_prefill(c.h, 0, lens, ntok, q, k, v, c.wq, c.wk, out)
        st, word = qa.qa_q4_get_device_error(c.h)
        assert st == 7 and word & 0xff == 1
        assert qa.qa_q4_get_device_error(c.h) == (0, 0)
        qa.qa_q4_prefill(c.h, 0, lens, ntok, q, k, v, c.wq, c.wk, out)
        assert qa.qa_q4_get_device_error(c.h) == (0, 0)
        qp, kp = c.transform(lens, ntok, q, k, v)
        c.note(0, lens, ntok, kp, f64(v))
        c.check_bytes()
        want, mag = c.want(lens, ntok, qp)
        close(out, want, mag, DECODE_BITS if kernel == 2 else PREFILL_BITS)
