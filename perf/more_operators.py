"""Cases of the 8-bit key/value cache: rows into the cache and back (append), a
decode step's attention over it (decode), a decode step that attends to a few
blocks which a cheap score picks for its queries (sparse), and prefill attention
against it, whole prompts or chunks (prefill).

The format.  A block is 64 consecutive positions of one kv head, from a multiple
of 64.  A block whose 64 rows have all been written is complete: its keys and its
values are each held as 64 x D integers n in -127..127 and one fp32 scale s, and
stand for n * s.  With a the largest magnitude of the block, s is a / 127 and n is
x * (127 / a) to the nearest integer, halves to even; the two quotients and the
product are fp32 numbers, rounded to nearest.  A block with a < 2^-64 holds zeros
(s = 0), one with a value that is not finite has s = NaN.  The rows of a block that
is not complete are held in bf16 as they came.  A call sees the rows that it brings
in bf16, and the complete blocks of the calls before it in 8 bits.

The score.  Of a complete block the smallest and the largest n of each dimension
are kept (lo, hi).  The queries of a kv head's group are made integers c in
-127..127 with one scale for the group, as above, and the block's score is
s * sum over the group's heads and the dimensions of max(c * lo, c * hi): as large
as their products with any key of the block can be together.  The first and the last
complete block, and those whose s is NaN, score infinity.  The n_blocks highest
scores are attended to, the lower index first among equals, and the rows of the
block that is not complete.

Where keys are normed they are RMS-normed per head and rotated before they are
written, queries before they attend, with the roundings of the framework's bf16
path: x_hat = bf16(x r), y = bf16(w x_hat), and one rounding of the rotated pair.

Where `own` is false the operators run in plain torch operations; where it is
true they are the framework's.
"""
import math

import torch

own = False

DEV = "cuda"
THETA, EPS = 1e6, 1e-6
BLOCK = 64
SMALL = 2.0 ** -64


# --------------------------------------------------------------------- cases
def _lens(text):
    return [int(x) for x in text.split(",")]


def _same(n, length):
    return ",".join([str(length)] * n)


def listed():
    return [
        # one new row for each of four sequences, of which every one completes a block
        dict(name="append_b4_t1", op="append", hq=32, hkv=8, d=128, start="511,1023,1535,2047", new="1,1,1,1"),
        # the rows of four prompts of mixed lengths, odd ranges behind what is there
        dict(name="append_ragged_prompts", op="append", hq=32, hkv=8, d=128, start="0,17,1,130",
             new="512,1023,1537,2048"),
        # a long context moved into the cache at once
        dict(name="append_b4_long", op="append", hq=32, hkv=8, d=128, start="0,0,0,0", new=_same(4, 16384)),
        # one token against a short cache: latency
        dict(name="decode_b1_l512", op="decode", norm=True, hq=32, hkv=8, d=128, start="512", new="1"),
        # the decode step of the four-prompt workload, at a block's last row; queries and keys come rotated
        dict(name="decode_b4_l2047", op="decode", norm=False, hq=32, hkv=8, d=128, start=_same(4, 2047), new="1,1,1,1"),
        # the longest caches of the decode sweep
        dict(name="decode_b4_l16384", op="decode", norm=True, hq=32, hkv=8, d=128, start=_same(4, 16384),
             new="1,1,1,1"),
        # many sequences of mixed lengths, head size 64, groups of eight query heads
        dict(name="decode_b24_ragged_d64", op="decode", norm=True, hq=32, hkv=4, d=64,
             start=",".join(str(1 + (i * 739) % 8191) for i in range(24)), new=_same(24, 1)),
        # one long conversation, a sixteenth of it attended to
        dict(name="sparse_b1_l16384", op="sparse", n_blocks=16, hq=32, hkv=8, d=128, start="16400", new="1"),
        # four contexts of four times the decode sweep's longest, a sixteenth of them
        dict(name="sparse_b4_l65536", op="sparse", n_blocks=64, hq=32, hkv=8, d=128, start="65536,65000,64001,60031",
             new="1,1,1,1"),
        # the prompt of the smallest workload
        dict(name="prefill_b1_p64", op="prefill", hq=2, hkv=1, d=64, start="0", new="64"),
        # four whole prompts
        dict(name="prefill_b4_p2048", op="prefill", hq=32, hkv=8, d=128, start="0,0,0,0", new=_same(4, 2048)),
        # the next chunk of two prompts behind what the cache holds, odd lengths
        dict(name="prefill_chunk_b2", op="prefill", hq=32, hkv=8, d=128, start="4099,1025", new="777,1001"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "sparse", "prefill"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 8])
    more = {}
    if op == "prefill":
        b = rng.randint(1, 4)
        g = min(g, 4)
        new = [_log(rng, 1, 900) for _ in range(b)]
        start = [0 if rng.random() < 0.4 else _log(rng, 1, 4000 if b <= 2 else 1500) for _ in range(b)]
    elif op == "append":
        b = _log(rng, 1, 6)
        new = [_log(rng, 1, 8192) for _ in range(b)]
        start = [0 if rng.random() < 0.4 else _log(rng, 1, 4000) for _ in range(b)]
    else:
        b = _log(rng, 1, 24 if op == "decode" else 8)
        new = [1] * b
        top = min(16384, 65536 // b) if op == "decode" else min(65536, 262144 // b)
        start = [_log(rng, 1, top) - 1 for _ in range(b)]
        more = {"norm": rng.random() < 0.6} if op == "decode" else {"n_blocks": _log(rng, 1, 64)}
    return dict(op=op, **more, hq=hkv * g, hkv=hkv, d=d, start=",".join(map(str, start)), new=",".join(map(str, new)))


def work(case):
    hq, hkv, d, op = case["hq"], case["hkv"], case["d"], case["op"]
    start, new = _lens(case["start"]), _lens(case["new"])
    tokens = sum(new)
    rows = 2 * tokens * hkv  # of K and V
    if op == "append":  # rows in, rows in 8 bits and their values out
        return {"bytes": rows * (2 * d + d + 2 * d), "flops": rows * d * 3}
    io = tokens * 2 * hq * d * 2 + rows * 2 * d  # q, out, k and v
    if op == "sparse":  # the bounds of every complete block, and the chosen ones
        full = [s // BLOCK for s in start]
        keys = [BLOCK * min(case["n_blocks"], f) + s % BLOCK + 1 for f, s in zip(full, start)]
        seen = sum(full) * hkv * (2 * d + 4) + 2 * sum(keys) * hkv * d
        return {"bytes": seen + io + rows * 2 * d, "flops": 4 * hq * d * sum(keys) + 4 * hkv * d * sum(full)}
    held = 2 * sum(start) * hkv * d  # read once: what the cache holds
    pairs = sum(n * s + n * (n + 1) // 2 for s, n in zip(start, new))
    values = rows * 2 * d if op == "decode" else rows * d + rows * d  # rows or values that come back, and the cache's
    return {"bytes": held + io + values, "flops": 4 * hq * d * pairs}


# -------------------------------------------------------------- the plain form
def _codes(x, dims):
    """Integers of x (fp32) with one scale over `dims`, and that scale."""
    a = x.abs().amax(dims, keepdim=True)
    fine = torch.isfinite(a)
    used = fine & (a >= SMALL)
    by = torch.full_like(a, 127.0) / torch.where(used, a, 1.0)  # by a tensor: true divisions
    n = torch.round(torch.where(used, x, 0.0) * by)
    s = torch.where(used, a / torch.full_like(a, 127.0), 0.0)
    return n, torch.where(fine, s, math.nan)


def _quantise(x):
    """Blocks x [..., 64, D] as int8 codes and scales [...]."""
    n, s = _codes(x.float(), (-2, -1))
    return n.to(torch.int8), s[..., 0, 0]


def _values(codes, scales):
    """fp32 values of blocks [Hkv, n, 64, D], as rows [Hkv, 64 n, D]."""
    return (codes.float() * scales[..., None, None]).flatten(1, 2)


def _norm_rope(x, w, pos):
    """x [T, H, D] at positions pos [T]: RMS norm, then the rotation of the halves."""
    d = x.shape[-1]
    f = x.float()
    r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    y = (w * (f * r).bfloat16()).float()
    ang = pos.double().unsqueeze(-1) * torch.pow(THETA, -2.0 * torch.arange(d // 2, device=x.device).double() / d)
    c, s = ang.cos().float().unsqueeze(1), ang.sin().float().unsqueeze(1)
    lo, hi = y[..., : d // 2], y[..., d // 2:]
    return torch.cat((lo * c - hi * s, hi * c + lo * s), -1).bfloat16()


def _plain_write(st, i, x):
    """Rows x [T, Hkv, D] into K (i = 0) or V (i = 1): blocks that are complete now
    as codes, the rest as it is."""
    for b, rows in enumerate(x.split(st["new"])):
        start, first = st["start"][b], st["start"][b] // BLOCK
        full = (start + rows.shape[0]) // BLOCK
        rows = torch.cat((st["old"][i][b], rows.transpose(0, 1)), 1)
        cut = (full - first) * BLOCK
        if cut:
            c, s = _quantise(rows[:, :cut].unflatten(1, (-1, BLOCK)))
            st["codes"][i][b, :, first:full], st["scales"][i][b, :, first:full] = c, s
            if i == 0:
                st["lo"][b, :, first:full], st["hi"][b, :, first:full] = c.amin(2), c.amax(2)
        st["tail"][i][b, :, : rows.shape[1] - cut] = rows[:, cut:]


def _plain_read(st, i):
    """The rows that the call wrote, as the cache holds them, bf16 [T, Hkv, D]."""
    got = []
    for b, (start, n) in enumerate(zip(st["start"], st["new"])):
        first, full = start // BLOCK, (start + n) // BLOCK
        rows = _values(st["codes"][i][b, :, first:full], st["scales"][i][b, :, first:full]).bfloat16()
        rows = torch.cat((rows, st["tail"][i][b, :, : (start + n) % BLOCK]), 1)
        got.append(rows[:, start % BLOCK:][:, :n].transpose(0, 1))
    return torch.cat(got)


def _plain_attend(st, q, k, v, blocks=None):
    """q [T, Hq, D] over the cache and the call's own rows k, v [T, Hkv, D] (all bf16
    values): causal softmax attention in fp32, over `blocks` alone where given."""
    hkv, d, outs, at = st["hkv"], st["d"], [], 0
    for b, (start, n) in enumerate(zip(st["start"], st["new"])):
        full = start // BLOCK
        held = []
        for i, x in enumerate((k, v)):
            c, s = st["codes"][i][b, :, :full], st["scales"][i][b, :, :full]
            if blocks is not None:
                pick = blocks[b].long().clamp(min=0)  # [Hkv, n_blocks]
                head = torch.arange(hkv, device=DEV).unsqueeze(1)
                c, s = st["codes"][i][b][head, pick], st["scales"][i][b][head, pick]
            own_rows = x[at:at + n].transpose(0, 1)
            held.append(torch.cat((_values(c, s), st["old"][i][b].float(), own_rows.float()), 1))
        qs = q[at:at + n].float().view(n, hkv, -1, d).permute(1, 2, 0, 3).flatten(1, 2)  # [Hkv, G n, D]
        t = torch.matmul(qs, held[0].transpose(-1, -2)) / math.sqrt(d)
        keys = t.shape[-1]
        unseen = torch.arange(keys, device=DEV) > torch.arange(keys - n, keys, device=DEV).unsqueeze(-1)
        t = t.unflatten(1, (-1, n)).masked_fill(unseen, -math.inf)
        if blocks is not None:  # places of the list that name no block
            none = torch.zeros(hkv, 1, 1, keys, device=DEV, dtype=torch.bool)
            cut = blocks.shape[-1] * BLOCK
            none[..., :cut] = (blocks[b] < 0).repeat_interleave(BLOCK, -1)[:, None, None]
            t = t.masked_fill(none, -math.inf)
            held[1] = torch.where(none[:, 0, 0].unsqueeze(-1), 0.0, held[1])
        p = torch.exp(t - t.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        o = torch.matmul(p.flatten(1, 2), held[1]).unflatten(1, (-1, n))  # [Hkv, G, n, D]
        outs.append(o.permute(2, 0, 1, 3).flatten(1, 2))
        at += n
    return torch.cat(outs).bfloat16()


def _plain_select(st, q):
    """Block indices int32 [B, Hkv, n_blocks] for queries q [B, Hq, D], ascending, -1 behind them."""
    b, hkv, n = len(st["new"]), st["hkv"], st["case"]["n_blocks"]
    c, _ = _codes(q.float().view(b, hkv, -1, st["d"]), (-2, -1))
    up, down = c.clamp(min=0).sum(2), c.clamp(max=0).sum(2)  # [B, Hkv, D]; all sums below stay under 2^24
    got = torch.full((b, hkv, n), -1, device=DEV, dtype=torch.int32)
    for i, start in enumerate(st["start"]):
        full = start // BLOCK
        if full == 0:
            continue
        s = st["scales"][0][i, :, :full]
        dot = (st["hi"][i, :, :full].float() * up[i].unsqueeze(1)).sum(-1)
        dot = dot + (st["lo"][i, :, :full].float() * down[i].unsqueeze(1)).sum(-1)
        score = dot * s
        score = torch.where(torch.isnan(s), math.inf, score)
        score[:, 0] = math.inf
        score[:, full - 1] = math.inf
        order = torch.sort(score, dim=-1, descending=True, stable=True).indices[:, :n]
        got[i, :, : order.shape[-1]] = order.sort(-1).values.int()
    return got


# ------------------------------------------------------------------- the states
def _rows(gen, shape, gain):
    return (torch.randn(shape, generator=gen, device=DEV) * gain).bfloat16()


def _inputs(case, seed):
    """What the seed gives: the rows that the cache holds before the call (per
    sequence, [start, Hkv, D]), the call's own, and the norm weights."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    start, new = _lens(case["start"]), _lens(case["new"])
    # Keys and values of a layer differ in size from channel to channel.
    gk = torch.exp(0.4 * torch.randn(hkv, d, generator=gen, device=DEV))
    gv = torch.exp(0.4 * torch.randn(hkv, d, generator=gen, device=DEV))
    t = sum(new)
    got = dict(k=_rows(gen, (t, hkv, d), gk), v=_rows(gen, (t, hkv, d), gv), wq=None, wk=None)
    if case["op"] != "append":
        got["q"] = _rows(gen, (t, hq, d), 1.0)
        if case["op"] == "prefill" or case.get("norm"):
            got["wq"] = (1 + 0.1 * torch.randn(d, generator=gen, device=DEV)).bfloat16()
            got["wk"] = (1 + 0.1 * torch.randn(d, generator=gen, device=DEV)).bfloat16()
    got["before"] = [tuple(_rows(gen, (s, hkv, d), gain) for gain in (gk, gv)) for s in start]
    return got


def prepare(case, seed):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    start, new = _lens(case["start"]), _lens(case["new"])
    n_blocks = case.get("n_blocks", 0)
    b, cap = len(new), max(max(s + n for s, n in zip(start, new)), BLOCK * n_blocks)
    got = _inputs(case, seed)
    before = got.pop("before")
    st = dict(got, case=case, op=case["op"], hq=hq, hkv=hkv, d=d, start=start, new=new)
    st["k_held"], st["v_held"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
    if "q" in st:
        st["out"] = torch.empty_like(st["q"])
    if n_blocks:
        st["blocks"] = torch.empty(b, hkv, n_blocks, device=DEV, dtype=torch.int32)
    if own:
        st["cache"] = _Cache(b, hq, hkv, d, cap)
        for i, (k, v) in enumerate(before):  # one sequence at a time: the others append nothing
            st["cache"].qa.qa_q8_append(st["cache"].handle, 0, [0] * b, [len(k) if j == i else 0 for j in range(b)], k, v)
        return st
    n = -(-cap // BLOCK)
    st["codes"] = [torch.zeros(b, hkv, n, BLOCK, d, device=DEV, dtype=torch.int8) for _ in range(2)]
    st["scales"] = [torch.zeros(b, hkv, n, device=DEV) for _ in range(2)]
    st["tail"] = [torch.zeros(b, hkv, BLOCK, d, device=DEV, dtype=torch.bfloat16) for _ in range(2)]
    st["lo"], st["hi"] = (torch.zeros(b, hkv, n, d, device=DEV, dtype=torch.int8) for _ in range(2))
    st["old"] = [[], []]  # rows of blocks that are not complete
    for j, kv in enumerate(before):
        full = start[j] // BLOCK
        for i, x in enumerate(kv):
            x = x.transpose(0, 1)
            st["old"][i].append(x[:, full * BLOCK:].contiguous())
            for lo in range(0, full, 256):  # a part at a time, for its fp32 copies
                hi = min(full, lo + 256)
                c, s = _quantise(x[:, lo * BLOCK:hi * BLOCK].unflatten(1, (-1, BLOCK)))
                st["codes"][i][j, :, lo:hi], st["scales"][i][j, :, lo:hi] = c, s
                if i == 0:
                    st["lo"][j, :, lo:hi], st["hi"][j, :, lo:hi] = c.amin(2), c.amax(2)
    st["pos"] = torch.cat([torch.arange(s, s + m, device=DEV) for s, m in zip(start, new)])
    return st


class _Cache:
    """The framework's 8-bit cache of one layer, freed with its state."""

    def __init__(self, b, hq, hkv, d, cap):
        from gqa_attention_preallocated_qa_gb300 import binding
        self.qa = binding
        self.handle = binding.qa_q8_cache_alloc(1, b, hq, hkv, d, cap, THETA, EPS)

    def __del__(self):
        if getattr(self, "handle", None):
            self.qa.qa_q8_cache_free(self.handle)


def run(st):
    op = st["op"]
    if own:
        qa, cache = st["cache"].qa, st["cache"].handle
        if op == "append":
            qa.qa_q8_append(cache, 0, st["start"], st["new"], st["k"], st["v"])
            qa.qa_q8_read(cache, 0, st["start"], st["new"], st["k_held"], st["v_held"])
            return {"k": st["k_held"], "v": st["v_held"]}
        if op == "decode":
            qa.qa_q8_decode_step(cache, 0, st["start"], st["q"], st["k"], st["v"], st["wq"], st["wk"], st["out"],
                                 st["k_held"], st["v_held"])
            return {"out": st["out"], "k": st["k_held"], "v": st["v_held"]}
        if op == "sparse":
            qa.qa_q8_sparse_step(cache, 0, st["start"], st["case"]["n_blocks"], st["q"], st["k"], st["v"], st["wq"],
                                 st["wk"], st["out"], st["blocks"], st["k_held"], st["v_held"])
            return {"out": st["out"], "blocks": st["blocks"], "k": st["k_held"], "v": st["v_held"]}
        qa.qa_q8_prefill(cache, 0, st["start"], st["new"], st["q"], st["k"], st["v"], st["wq"], st["wk"], st["out"])
        # The appended values come back too.  (V only: of millions of rotated keys a
        # few lie so near a border of bf16 that two right programs round them apart.)
        qa.qa_q8_read(cache, 0, st["start"], st["new"], None, st["v_held"])
        return {"out": st["out"], "v": st["v_held"]}
    q, k, v = st.get("q"), st["k"], st["v"]
    if st["wq"] is not None:
        q, k = _norm_rope(q, st["wq"], st["pos"]), _norm_rope(k, st["wk"], st["pos"])
    blocks = _plain_select(st, q) if op == "sparse" else None
    out = _plain_attend(st, q, k, v, blocks) if op != "append" else None
    _plain_write(st, 0, k)
    _plain_write(st, 1, v)
    if op == "append":
        return {"k": _plain_read(st, 0), "v": _plain_read(st, 1)}
    if op == "prefill":
        return {"out": out, "v": _plain_read(st, 1)}
    # A step's own rows, as it attended to them.
    return {"out": out, "blocks": blocks, "k": k, "v": v} if op == "sparse" else {"out": out, "k": k, "v": v}


# ------------------------------------------------------------------ in 64 bits
def _exact_codes(x):
    """Integers and the scale of all of x [Hkv, ..., D], one scale for each of [Hkv, ...]'s
    leading index, from the definition: fp32 quotients, taken from 64-bit ones."""
    f = x.double().flatten(1)
    top = f.abs().max(1).values
    by = (127.0 / top.clamp(min=SMALL)).float().double()
    n = (f * by[:, None]).float().double().round()
    s = (top / 127.0).float().double()
    small = top < SMALL
    return torch.where(small[:, None], 0.0, n).view(x.shape), torch.where(small, 0.0, s)


def _exact_blocks(rows, full):
    """Codes [Hkv, full, 64, D] and scales [Hkv, full] of rows [n, Hkv, D]'s first blocks."""
    x = rows[: full * BLOCK].transpose(0, 1).reshape(rows.shape[1], full, BLOCK, rows.shape[2])
    n, s = _exact_codes(x.flatten(0, 1))
    return n.view(x.shape), s.view(x.shape[:2])


def _exact_norm_rope(x, w, first):
    n, _, d = x.shape
    f = x.double()
    hat = (f / torch.sqrt((f * f).sum(-1, keepdim=True) / d + EPS)).bfloat16().double()
    y = (w.double() * hat).bfloat16().double()
    pos = torch.arange(first, first + n, device=DEV).double()
    i = torch.arange(d // 2, device=DEV).double()
    ang = pos[:, None] * torch.exp(-2.0 * i / d * math.log(THETA))[None]
    z = torch.complex(y[..., : d // 2], y[..., d // 2:]) * torch.polar(torch.ones_like(ang), ang)[:, None]
    return torch.cat((z.real, z.imag), -1).bfloat16()


def _exact_select(q, k_rows, full, n_blocks):
    """Ascending lists [Hkv, n_blocks] of the chosen blocks, by the products themselves."""
    hkv = k_rows.shape[1]
    got = torch.full((hkv, n_blocks), -1, device=DEV, dtype=torch.int32)
    if full == 0:
        return got
    c, _ = _exact_codes(q.view(hkv, -1, q.shape[-1]))
    n, s = _exact_blocks(k_rows, full)
    least, most = n.min(2).values, n.max(2).values  # [Hkv, full, D]
    for h in range(hkv):
        each = torch.maximum(c[h][:, None] * least[h], c[h][:, None] * most[h])  # [G, full, D]
        score = (each.sum((0, 2)) * s[h]).float()  # one rounding, as s is fp32 and the sum an integer below 2^24
        score[0] = score[-1] = math.inf
        rank = sorted(range(full), key=lambda j, x=score.tolist(): (-x[j], j))[:n_blocks]
        got[h, : len(rank)] = torch.tensor(sorted(rank), dtype=torch.int32)
    return got


def exact(case, seed):
    hq, hkv, d, op = case["hq"], case["hkv"], case["d"], case["op"]
    start, new = _lens(case["start"]), _lens(case["new"])
    got = _inputs(case, seed)
    outs, lists, ks, vs, at = [], [], [], [], 0
    for i, (s, n) in enumerate(zip(start, new)):
        rows = [got["k"][at:at + n], got["v"][at:at + n]]
        q = got["q"][at:at + n] if op != "append" else None
        if got["wq"] is not None:
            q, rows[0] = _exact_norm_rope(q, got["wq"], s), _exact_norm_rope(rows[0], got["wk"], s)
        if op != "append":
            full = s // BLOCK
            if op == "sparse":
                lists.append(_exact_select(q[0], got["before"][i][0], full, case["n_blocks"]))
            o = torch.empty(n, hq, d, dtype=torch.float64, device=DEV)
            for h in range(hkv):
                pick = [j for j in lists[-1][h].tolist() if j >= 0] if op == "sparse" else list(range(full))
                both = []
                for x, mine in zip(got["before"][i], rows):
                    blocks = x[: full * BLOCK, h].view(full, BLOCK, d)[pick]  # the chosen ones [.., 64, D]
                    codes, scales = _exact_codes(blocks) if pick else (blocks.double(), x.new_zeros(0).double())
                    held = (codes * scales[:, None, None]).reshape(-1, d)
                    both.append(torch.cat((held, x[full * BLOCK:, h].double(), mine[:, h].double())))
                keys = both[0].shape[0]
                unseen = torch.arange(keys, device=DEV)[None] > torch.arange(keys - n, keys, device=DEV)[:, None]
                for j in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                    logit = q[:, j].double() @ both[0].T / math.sqrt(d)
                    o[:, j] = torch.softmax(logit.masked_fill(unseen, -math.inf), -1) @ both[1]
            outs.append(o)
        if op in ("append", "prefill"):  # what the cache then holds of the new rows
            for x, mine, held in zip(got["before"][i], rows, (ks, vs)):
                x = torch.cat((x[s // BLOCK * BLOCK:], mine))
                full = len(x) // BLOCK
                done = x[:0].double()
                if full:
                    codes, scales = _exact_blocks(x, full)
                    done = (codes * scales[..., None, None]).flatten(1, 2).transpose(0, 1)
                held.append(torch.cat((done, x[full * BLOCK:].double()))[s % BLOCK:])
        else:
            ks.append(rows[0])
            vs.append(rows[1])
        at += n
    k, v = torch.cat(ks).double(), torch.cat(vs).double()
    if op == "append":
        return {"k": k, "v": v}
    out = torch.cat(outs)
    if op == "sparse":
        return {"out": out, "blocks": torch.stack(lists), "k": k, "v": v}
    return {"out": out, "k": k, "v": v} if op == "decode" else {"out": out, "v": v}
