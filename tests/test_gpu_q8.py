"""The 8-bit cache on the GPU against its definition (q8_ref.py).

Tolerances, from the roundings alone.  A decode step multiplies the codes themselves,
which fp16 holds, with queries scaled by a power of two, which fp16 holds down to 2^-22
of a row's largest value.  The weights P are rounded to fp16, relative to a reference
that is at most 2^8 below the largest: 2^-11 of a weight, or 2^-25 of the largest weight where
that is more.  Scores are fp32 sums in which every code carries 128 that is taken
away again: with terms below 2^-24 (2^8 + 2^7) of the largest query, 8 sums of 2^-23 each,
that is below 2^-13 of a weight for the queries and keys here (sum |q| below 2^7, s below 2^-4,
log2(e) / sqrt(D) below 0.19).  Numerator and denominator use the same weights, so an
output moves by at most 2 (2^-11 + 2^-13) sum p |v| + 2^-24 sum |v| / l, and then one
rounding to bf16, 2^-8 |out|.  The bf16 rows' weights are sums of two bf16 numbers (2^-16),
inside that bound.  The prefill kernel rounds P to bf16: 2^-8 in the place of 2^-11.
"""
import numpy as np
import pytest
import torch

import q8_ref
from gpu_util import f64

pytestmark = pytest.mark.gpu

THETA, EPS = 1e6, 1e-6
BLOCK = q8_ref.BLOCK


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
    """An 8-bit cache of one layer beside what it should hold."""

    def __init__(self, qa, batch, hq, hkv, d, cap, layers=1, seed=1):
        self.qa, self.hq, self.hkv, self.d, self.cap, self.batch = qa, hq, hkv, d, cap, batch
        self.h = qa.qa_q8_cache_alloc(layers, batch, hq, hkv, d, cap, THETA, EPS)
        self.ref = q8_ref.Rows(batch, hkv, d, cap)
        self.wq, self.wk = 1 + 0.1 * rows(seed, d), 1 + 0.1 * rows(seed + 1, d)

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.qa.qa_q8_cache_free(self.h)

    def append(self, start, ntok, k, v, layer=0):
        self.qa.qa_q8_append(self.h, layer, start, ntok, k, v)
        self.ref.write(start, ntok, f64(k), f64(v))

    def fill(self, lens, seed, gain=1.0):
        k, v = rows(seed, sum(lens), self.hkv, self.d, gain=gain), rows(seed + 1, sum(lens), self.hkv, self.d)
        self.append([0] * len(lens), lens, k, v)

    def check_read(self, lens, start=None, ntok=None, layer=0):
        start = start or [0] * len(lens)
        ntok = ntok or [n - s for n, s in zip(lens, start)]
        k = torch.full((sum(ntok), self.hkv, self.d), 7.0, device="cuda", dtype=torch.bfloat16)
        v = k.clone()
        self.qa.qa_q8_read(self.h, layer, start, ntok, k, v)
        at = 0
        for b, (s, n) in enumerate(zip(start, ntok)):
            for i, x in enumerate((k, v)):
                np.testing.assert_array_equal(f64(x[at:at + n]), self.ref.read(i, b, s, n, lens[b]), err_msg=f"sequence {b}, {'kv'[i]}")
            at += n

    def tokens(self, n, seed):
        return rows(seed, n, self.hq, self.d), rows(seed + 1, n, self.hkv, self.d), rows(seed + 2, n, self.hkv, self.d)

    def want(self, b, pos, q, blocks=None):
        """Attention of q [1, Hq, D] (float64) at position pos, whose row the reference has."""
        full = pos // BLOCK
        outs, mags, flats = [], [], []
        g = self.hq // self.hkv
        k, v = (self.ref.held(i, b, pos, blocks) for i in (0, 1))
        for h in range(self.hkv):
            kk, vv = (torch.from_numpy(np.concatenate((x[h], self.ref.came[i, b, h, pos:pos + 1]))).cuda()[None]
                      for i, x in enumerate((k, v)))
            o, m, f = q8_ref.attend(q[:, h * g:(h + 1) * g], kk, vv, kk.shape[1] - 1)
            outs.append(o)
            mags.append(m)
            flats.append(f)
        assert full == pos // BLOCK
        return torch.cat(outs, 1), torch.cat(mags, 1), torch.cat(flats, 1)


def close(got, want, mag, flat, p_bits=11, what=""):
    got = got.double()
    tol = 2.0 ** -8 * want.abs() + 2 * (2.0 ** -p_bits + 2.0 ** -13) * mag + 2.0 ** -24 * flat + 1e-6
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {float(((got - want).abs() / tol).max()):.3f} of the tolerance"


# ------------------------------------------------------------------ rows
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv", [1, 3])
def test_append_and_read_are_the_definition(qa, d, hkv):
    lens = [64, 1, 63, 65, 200, 128, 0, 513]
    with Cache(qa, len(lens), 2 * hkv, hkv, d, 520) as c:
        c.fill(lens, 5)
        c.check_read(lens)
        c.check_read(lens, [10, 0, 62, 64, 63, 0, 0, 449], [50, 1, 1, 1, 66, 128, 0, 64])


@pytest.mark.parametrize("d", [64, 128])
def test_what_is_held_does_not_depend_on_the_calls(qa, d):
    lens, cuts = [300, 129, 64], [[1, 62, 1, 3, 61, 70, 102], [64, 64, 1], [63, 1]]
    k, v = rows(1, sum(lens), 2, d), rows(2, sum(lens), 2, d)
    offs = np.cumsum([0] + lens)
    with Cache(qa, 3, 4, 2, d, 320) as c:
        at = [0, 0, 0]
        for step in range(7):
            n = [cut[step] if step < len(cut) else 0 for cut in cuts]
            part = [x for b in range(3) for x in range(offs[b] + at[b], offs[b] + at[b] + n[b])]
            c.append(at, n, k[part].contiguous(), v[part].contiguous())
            at = [a + m for a, m in zip(at, n)]
            c.check_read(at)
        assert at == lens


@pytest.mark.parametrize("d", [64, 128])
def test_blocks_of_every_size_of_number(qa, d):
    """Largest magnitudes over bf16's range, ties, zeros, values below 2^-64, and some
    that are not finite: each in a block of its own."""
    rng = np.random.default_rng(d)
    tops = [2.0 ** e for e in range(-126, 127, 11)] + [0.0, 2.0 ** -64, 2.0 ** -65 * 1.9921875, 3.3895e38, 127.0, 254.0]
    x = rng.uniform(-1, 1, (len(tops) + 3, BLOCK, 1, d)).astype(np.float32)
    halves = (rng.integers(-126, 127, x.shape) + 0.5).astype(np.float32) / 127  # a tie where the scale is a power of two / 127
    x = np.where(rng.random(x.shape) < 0.5, x, halves)
    x[:, 5, 0, 3] = 1.0
    for i, top in enumerate(tops):
        x[i] *= np.float32(top)
    x[len(tops), 63, 0, d - 1] = np.nan
    x[len(tops) + 1, 0, 0, 0] = np.inf
    x[len(tops) + 2, 17, 0, 9] = -np.inf
    n = x.shape[0] * BLOCK
    k = torch.from_numpy(x.reshape(n, 1, d)).cuda().bfloat16()
    with Cache(qa, 1, 1, 1, d, n + 3) as c:
        c.append([0], [n], k, k.flip(0).contiguous())
        c.check_read([n])


def test_ranges_elsewhere_are_left_alone(qa):
    with Cache(qa, 3, 4, 2, 128, 256, layers=2) as c:
        c.fill([100, 256, 31], 3)
        k, v = rows(9, 5, 2, 128), rows(10, 5, 2, 128)
        qa.qa_q8_append(c.h, 1, [0, 0, 0], [2, 0, 3], k, v)  # another layer
        c.check_read([100, 256, 31])
        c.append([100, 0, 0], [5, 0, 0], k, v)  # sequences with nothing new
        c.check_read([105, 256, 31])
        ko = torch.zeros(5, 2, 128, device="cuda", dtype=torch.bfloat16)
        qa.qa_q8_read(c.h, 1, [0, 0, 0], [2, 0, 3], ko, None)
        assert torch.equal(ko, k)


# ------------------------------------------------------------------ decode
GEOMETRIES = [(1, 1, 64), (8, 1, 128), (4, 2, 64), (6, 6, 128), (16, 8, 128), (32, 8, 128), (32, 4, 64)]


@pytest.mark.parametrize("hq,hkv,d", GEOMETRIES)
def test_decode_is_attention_over_what_is_held(qa, hq, hkv, d):
    lens = [0, 1, 63, 64, 65, 127, 128, 700, 1500]
    with Cache(qa, len(lens), hq, hkv, d, 1600) as c:
        c.fill(lens, 11)
        q, k, v = c.tokens(len(lens), 21)
        out = torch.full_like(q, 9.0)
        kh, vh = torch.empty_like(k), torch.empty_like(v)
        qa.qa_q8_decode_step(c.h, 0, lens, q, k, v, None, None, out, kh, vh)
        assert torch.equal(kh, k) and torch.equal(vh, v)
        c.ref.write(lens, [1] * len(lens), f64(k), f64(v))
        for b, pos in enumerate(lens):
            close(out[b:b + 1], *c.want(b, pos, q[b:b + 1].double()), what=f"position {pos}")
        c.check_read([n + 1 for n in lens])
        assert qa.qa_q8_get_device_error(c.h)[0] == 0


@pytest.mark.parametrize("blocks", [0, 2])
@pytest.mark.parametrize("q_size,k_size", [(2.0 ** -120, 2.0 ** 120), (2.0 ** 60, 2.0 ** -60)])
def test_scores_of_ordinary_size_from_queries_and_keys_that_are_not(qa, q_size, k_size, blocks):
    """A query row of 2^-120 is scaled by 2^115 at most, so fp16 holds it in steps of 2^-139: half
    a step of 2^-19 of such a value, 128 times, against keys below 5 and log2(e) / sqrt(D) = 0.1275,
    moves a score by less than 2^-13; 2^-11 + 2 * 2^-13 is below 2^-10."""
    hq, hkv, d, pos = 8, 2, 128, 300
    with Cache(qa, 1, hq, hkv, d, 400) as c:
        k, v = rows(1, pos, hkv, d), rows(2, pos, hkv, d)
        c.append([0], [pos], k * k_size, v)
        q, nk, nv = rows(3, 1, hq, d) * q_size, rows(4, 1, hkv, d) * k_size, rows(5, 1, hkv, d)
        out = torch.empty_like(q)
        lists = torch.empty(1, hkv, max(blocks, 1), dtype=torch.int32, device="cuda")
        if blocks:
            qa.qa_q8_sparse_step(c.h, 0, [pos], blocks, q, nk, nv, None, None, out, lists)
        else:
            qa.qa_q8_decode_step(c.h, 0, [pos], q, nk, nv, None, None, out)
        c.ref.write([pos], [1], f64(nk), f64(nv))
        close(out, *c.want(0, pos, q.double(), lists[0].cpu().numpy() if blocks else None), p_bits=10)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_steps_follow_each_other_through_blocks(qa, d):
    lens = [60, 126, 0]
    with Cache(qa, 3, 8, 2, d, 512) as c:
        c.fill(lens, 31)
        for step in range(70):
            q, k, v = c.tokens(3, 100 + 3 * step)
            out = torch.empty_like(q)
            qa.qa_q8_decode_step(c.h, 0, lens, q, k, v, None, None, out)
            c.ref.write(lens, [1, 1, 1], f64(k), f64(v))
            if step % 9 < 6:
                for b, pos in enumerate(lens):
                    close(out[b:b + 1], *c.want(b, pos, q[b:b + 1].double()), what=f"step {step}, position {pos}")
            lens = [n + 1 for n in lens]
        c.check_read(lens)


def transform(qa, c, start, ntok, q, k, v):
    """q', k' of the bf16 path's kernel for prompts, as bf16 tensors."""
    bf16 = qa.qa_cache_alloc(1, c.batch, c.hq, c.hkv, c.d, c.cap, THETA, EPS)
    try:
        kt, _, _ = qa.cache_tensors(bf16, 0, c.batch, c.hkv, c.cap, c.d)
        qa.qa_cache_set_lengths(bf16, 0, list(start) + [0] * (c.batch - len(start)))
        qp = torch.empty_like(q)
        qa.qa_prefill_transform(bf16, 0, list(ntok), q, k, v, c.wq, c.wk, qp)
        kp = torch.cat([kt[b, :, s:s + n].transpose(0, 1) for b, (s, n) in enumerate(zip(start, ntok))])
        return qp, kp.contiguous()
    finally:
        qa.qa_cache_free(bf16)


@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (32, 8, 128)])
def test_norm_and_rotation_inside_the_step(qa, hq, hkv, d):
    """The step gives the same bits for raw rows as for rows that another kernel normed."""
    lens = [0, 5, 63, 300]
    with Cache(qa, 4, hq, hkv, d, 400) as c, Cache(qa, 4, hq, hkv, d, 400) as other:
        c.fill(lens, 3)
        other.fill(lens, 3)
        q, k, v = c.tokens(4, 50)
        qp, kp = transform(qa, c, lens, [1] * 4, q, k, v)
        outs, held = [], []
        for cache, x, y, w in ((c, q, k, (c.wq, c.wk)), (other, qp, kp, (None, None))):
            out, kh, vh = torch.empty_like(q), torch.empty_like(k), torch.empty_like(k)
            qa.qa_q8_decode_step(cache.h, 0, lens, x, y, v, *w, out, kh, vh)
            outs.append(out)
            held.append(kh)
        assert torch.equal(held[0], kp) and torch.equal(held[1], kp)
        assert torch.equal(outs[0], outs[1])


# ------------------------------------------------------------------ sparse steps
def check_sparse(qa, c, lens, n_blocks, seed, gain=1.0):
    q, k, v = c.tokens(len(lens), seed)
    q = q * gain
    out = torch.empty_like(q)
    blocks = torch.full((len(lens), c.hkv, n_blocks), 12345, device="cuda", dtype=torch.int32)
    qa.qa_q8_sparse_step(c.h, 0, lens, n_blocks, q, k, v, None, None, out, blocks)
    got = blocks.cpu().numpy()
    c.ref.write(lens, [1] * len(lens), f64(k), f64(v))
    g = c.hq // c.hkv
    for b, pos in enumerate(lens):
        qs = f64(q[b]).reshape(c.hkv, g, c.d)
        for h in range(c.hkv):
            full = pos // BLOCK
            want = q8_ref.select(qs[h], c.ref.n[0, b, h, :full], c.ref.s[0, b, h, :full], n_blocks)
            np.testing.assert_array_equal(got[b, h], want, err_msg=f"position {pos}, kv head {h}")
        close(out[b:b + 1], *c.want(b, pos, q[b:b + 1].double(), got[b]), what=f"position {pos}")
    return [n + 1 for n in lens]


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (8, 1, 128), (32, 8, 128), (8, 4, 64)])
@pytest.mark.parametrize("n_blocks", [1, 2, 5, 16])
def test_sparse_step_is_the_definition(qa, hq, hkv, d, n_blocks):
    lens = [0, 63, 64, 65, 128, 319, 1000, 2047]
    with Cache(qa, len(lens), hq, hkv, d, 2100) as c:
        c.fill(lens, 7)
        for step in range(2):
            lens = check_sparse(qa, c, lens, n_blocks, 70 + 3 * step)


def test_sparse_choice_among_equal_scores(qa):
    """Blocks that are copies of each other: the lower index first; zeros; a block of NaN."""
    d, hkv, full = 64, 2, 40
    block = rows(1, BLOCK, hkv, d)
    k = block.repeat(full, 1, 1)
    k[BLOCK * 7:BLOCK * 9] = 0
    k[BLOCK * 20 + 3, 1, 5] = float("nan")  # of one kv head
    v = rows(2, full * BLOCK, hkv, d)
    with Cache(qa, 1, 4, hkv, d, full * BLOCK + 5) as c:
        c.append([0], [full * BLOCK], k, v)
        q, kn, vn = c.tokens(1, 9)
        out, blocks = torch.empty_like(q), torch.empty(1, hkv, 6, device="cuda", dtype=torch.int32)
        qa.qa_q8_sparse_step(c.h, 0, [full * BLOCK], 6, q, kn, vn, None, None, out, blocks)
        assert blocks[0, 0].tolist() == [0, 1, 2, 3, 4, 39]
        assert blocks[0, 1].tolist() == [0, 1, 2, 3, 20, 39]
        assert torch.isfinite(out[0, :2]).all() and torch.isnan(out[0, 2:]).all()
        # queries of zeros: every score is zero
        qa.qa_q8_sparse_step(c.h, 0, [full * BLOCK], 4, torch.zeros_like(q), kn, vn, None, None, out, blocks[:, :, :4].contiguous())
        z = torch.empty(1, hkv, 4, device="cuda", dtype=torch.int32)
        qa.qa_q8_sparse_step(c.h, 0, [full * BLOCK], 4, torch.zeros_like(q), kn, vn, None, None, out, z)
        assert z[0, 0].tolist() == [0, 1, 2, 39] and z[0, 1].tolist() == [0, 1, 20, 39]


@pytest.mark.parametrize("n_blocks", [1, 300, 2500])
def test_sparse_over_the_longest_cache(qa, n_blocks):
    """16384 blocks, more than the threads keep in registers."""
    cap, d = 1 << 20, 64
    gen = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn(cap - 1, 1, d, generator=gen, device="cuda").bfloat16()
    with Cache(qa, 1, 2, 1, d, cap) as c:
        c.append([0], [cap - 1], k, k)
        check_sparse(qa, c, [cap - 1], n_blocks, 5)


@pytest.mark.parametrize("d,n_blocks", [(128, 16382), (64, 16384)])
def test_sparse_with_the_largest_lists(qa, d, n_blocks):
    """16383 complete blocks: all but one of them, and all."""
    cap = 1 << 20
    k = rows(1, cap - 1, 1, d)
    with Cache(qa, 1, 8, 1, d, cap) as c:
        c.append([0], [cap - 1], k, k)
        check_sparse(qa, c, [cap - 1], n_blocks, 5)


# ------------------------------------------------------------------ prefill
def check_prefill(qa, c, start, ntok, seed):
    t = sum(ntok)
    q, k, v = c.tokens(t, seed)
    out = torch.empty_like(q)
    qa.qa_q8_prefill(c.h, 0, start, ntok, q, k, v, c.wq, c.wk, out)
    qp, kp = transform(qa, c, start, ntok, q, k, v)
    g, at = c.hq // c.hkv, 0
    for b, (s, n) in enumerate(zip(start, ntok)):
        if n == 0:
            continue
        outs, mags, flats = [], [], []
        for h in range(c.hkv):
            kk, vv = (torch.cat((torch.from_numpy(c.ref.held(i, b, s)[h]).cuda(), x[at:at + n, h].double()))[None]
                      for i, x in enumerate((kp, v)))
            o, m, f = q8_ref.attend(qp[at:at + n, h * g:(h + 1) * g].double(), kk, vv, s)
            outs.append(o)
            mags.append(m)
            flats.append(f)
        close(out[at:at + n], torch.cat(outs, 1), torch.cat(mags, 1), torch.cat(flats, 1), p_bits=8,
              what=f"{n} tokens at {s}")
        at += n
    c.ref.write(start, ntok, f64(kp), f64(v))
    return [s + n for s, n in zip(start, ntok)]


@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 64), (4, 4, 128), (32, 8, 128), (16, 2, 64)])
def test_prefill_of_prompts_and_chunks(qa, hq, hkv, d):
    with Cache(qa, 4, hq, hkv, d, 1200) as c:
        lens = check_prefill(qa, c, [0, 0, 0, 0], [130, 1, 64, 0], 40)
        lens = check_prefill(qa, c, lens, [500, 63, 129, 5], 50)
        lens = check_prefill(qa, c, lens, [1, 64, 300, 59], 60)
        c.check_read(lens)
        assert qa.qa_q8_get_device_error(c.h)[0] == 0


def test_prefill_of_few_blocks_behind_many_keys(qa):
    """Keys in parts, and the same with a sequence that has nothing before it."""
    with Cache(qa, 2, 16, 2, 128, 5000) as c:
        c.fill([4500, 0], 3)
        lens = check_prefill(qa, c, [4500, 0], [100, 70], 40)
        assert qa.qa_q8_stats(c.h)["prefill_attn"] == 1
        check_prefill(qa, c, lens, [70, 0], 50)


def test_prefill_of_more_sequences_than_the_workspace_holds(qa):
    n = 11
    with Cache(qa, n, 4, 1, 64, 300) as c:
        start = [(37 * i) % 150 for i in range(n)]
        c.fill(start, 3)
        lens = check_prefill(qa, c, start, [(53 * i) % 140 for i in range(n)], 40)
        c.check_read(lens)


def test_prefill_behind_values_of_every_size(qa):
    """Blocks of zeros, of large and of small values before a chunk: their scales are
    factors of the attention kernel's weights."""
    d, n = 128, 6 * BLOCK
    v = rows(1, n, 1, d)
    for j, size in enumerate([0.0, 2.0 ** 40, 2.0 ** -40, 2.0 ** -63, 1.0, 2.0 ** 100]):
        v[j * BLOCK:(j + 1) * BLOCK] *= size
    k = rows(2, n, 1, d)
    k[BLOCK:2 * BLOCK] = 0
    with Cache(qa, 1, 4, 1, d, 600) as c:
        for last in (5, 6):  # with and without the largest
            c.append([0], [last * BLOCK], k[:last * BLOCK].contiguous(), v[:last * BLOCK].contiguous())
            check_prefill(qa, c, [last * BLOCK], [70], 40)


# ------------------------------------------------------------------ all of it as it is used
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (4, 2, 64)])
def test_a_conversation(qa, hq, hkv, d):
    with Cache(qa, 3, hq, hkv, d, 1500) as c:
        lens = check_prefill(qa, c, [0, 0, 0], [600, 130, 1], 40)
        for turn in range(2):
            for step in range(5):
                q, k, v = c.tokens(3, 500 + 50 * turn + 3 * step)
                out, kh, vh = torch.empty_like(q), torch.empty_like(k), torch.empty_like(k)
                qa.qa_q8_decode_step(c.h, 0, lens, q, k, v, c.wq, c.wk, out, kh, vh)
                qp, kp = transform(qa, c, lens, [1] * 3, q, k, v)
                assert torch.equal(kh, kp) and torch.equal(vh, v)
                c.ref.write(lens, [1] * 3, f64(kp), f64(v))
                for b, pos in enumerate(lens):
                    close(out[b:b + 1], *c.want(b, pos, qp[b:b + 1].double()), what=f"position {pos}")
                lens = [n + 1 for n in lens]
            lens = check_sparse(qa, c, lens, 3, 700 + turn)
            lens = check_prefill(qa, c, lens, [60, 128, 200], 800 + 10 * turn)
        c.check_read(lens)
