"""Cases of the 4-bit key/value cache: quantising rows as they are written
(append), reading them back (read), a decode step's attention over the cache
(decode), and prefill attention against it, whole prompts or chunks (prefill).

The format.  A row (one position of one kv head, D = 64 or 128 values) is cut
into groups of 32 consecutive dimensions.  A group has one scale byte and 32
codes of 4 bits; it stands for the values (n - 8) * s, n in 0..15.  The scale
byte is the upper byte of an fp16 number (5 exponent bits, 2 mantissa bits):
s is max|x| / 7 rounded to the nearest such number (ties to even), at most 56.
n - 8 is x / s rounded to the nearest integer, halves away from zero, held to
-8..7; a scale of zero gives n = 8.  A group with a value that is not finite
has the scale byte 0x7f (NaN) and codes 8.  Byte i of a row's codes holds
dimension 2i in its low half and 2i + 1 in its high half.  A value has at most
7 significant bits, so bf16 holds every one exactly.

Keys are RMS-normed per head and rotated before they are quantised, queries
before they attend, with the roundings of the framework's bf16 path:
x_hat = bf16(x r), y = bf16(w x_hat), and one rounding of the rotated pair.
The new tokens' own keys and values are attended to as the cache holds them.

Where `own` is false the operators run in plain torch operations; where it is
true they are the framework's.
"""
import math

import torch

own = False

DEV = "cuda"
THETA, EPS = 1e6, 1e-6


# --------------------------------------------------------------------- cases
def _lens(text):
    return [int(x) for x in text.split(",")]


def _same(n, length):
    return ",".join([str(length)] * n)


def listed():
    return [
        # one new row for each of four sequences: the smallest write, all latency
        dict(name="append_b4_t1", op="append", hq=32, hkv=8, d=128, start="511,1023,1535,2047", new="1,1,1,1"),
        # the rows of four prompts of mixed lengths
        dict(name="append_ragged_prompts", op="append", hq=32, hkv=8, d=128, start="0,0,0,0", new="512,1024,1536,2048"),
        # a long context moved into the cache at once, odd ranges
        dict(name="append_b4_long", op="append", hq=32, hkv=8, d=128, start="0,17,1,130", new="16384,16301,8191,16383"),
        # a short cache of head size 64 read back
        dict(name="read_b1_l512_d64", op="read", hq=8, hkv=4, d=64, start="0", new="512"),
        # a long cache read back (moved to another form, or to another place)
        dict(name="read_b4_l16384", op="read", hq=32, hkv=8, d=128, start="0,0,0,0", new=_same(4, 16384)),
        # one token against a short cache: latency
        dict(name="decode_b1_l512", op="decode", hq=32, hkv=8, d=128, start="512", new="1"),
        # the decode step of the four-prompt workload
        dict(name="decode_b4_l2048", op="decode", hq=32, hkv=8, d=128, start=_same(4, 2048), new="1,1,1,1"),
        # the longest caches of the decode sweep
        dict(name="decode_b4_l16384", op="decode", hq=32, hkv=8, d=128, start=_same(4, 16384), new="1,1,1,1"),
        # many sequences of mixed lengths, head size 64, groups of eight query heads
        dict(name="decode_b24_ragged_d64", op="decode", hq=32, hkv=4, d=64,
             start=",".join(str(1 + (i * 739) % 8191) for i in range(24)), new=_same(24, 1)),
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
    op = rng.choice(["append", "read", "decode", "prefill"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 8])
    if op == "prefill":
        b = rng.randint(1, 4)
        g = min(g, 4)
        new = [_log(rng, 1, 900) for _ in range(b)]
        start = [0 if rng.random() < 0.4 else _log(rng, 1, 4000 if b <= 2 else 1500) for _ in range(b)]
    elif op == "decode":
        b = _log(rng, 1, 24)
        new = [1] * b
        top = min(16384, 65536 // b)
        start = [_log(rng, 1, top) - 1 for _ in range(b)]
    else:
        b = _log(rng, 1, 6)
        new = [_log(rng, 1, 8192) for _ in range(b)]
        start = [0 if rng.random() < 0.4 else _log(rng, 1, 4000) for _ in range(b)]
    return dict(op=op, hq=hkv * g, hkv=hkv, d=d, start=",".join(map(str, start)), new=",".join(map(str, new)))


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    start, new = _lens(case["start"]), _lens(case["new"])
    tokens, row4 = sum(new), d // 2 + d // 32
    rows = 2 * tokens * hkv  # of K and V
    if case["op"] == "append":  # rows in, rows in 4 bits and their values out
        return {"bytes": rows * (2 * d + row4 + 2 * d), "flops": rows * d * 4}
    if case["op"] == "read":
        return {"bytes": rows * (row4 + 2 * d), "flops": rows * d * 2}
    held = 2 * sum(start) * hkv * row4  # read once: what the cache holds
    pairs = sum(n * s + n * (n + 1) // 2 for s, n in zip(start, new))
    io = tokens * (2 * hq + 2 * hkv) * d * 2 + 4 * d + rows * row4
    values = rows * 2 * d if case["op"] == "decode" else rows * d  # the appended values that come back
    return {"bytes": held + io + values, "flops": 4 * hq * d * pairs}


# -------------------------------------------------------------- the plain form
def _quantise(x):
    """Codes and scale bytes of rows x [..., D], in fp32: every division below is
    of bf16 values, so a quotient that is a half or a midpoint is exact and any
    other is further from it than fp32's rounding."""
    g = x.float().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    a = g.abs().amax(-1, keepdim=True)
    fine = torch.isfinite(a)
    a = torch.where(fine, a, 0.0)
    t = (a / torch.full_like(a, 7.0)).clamp(max=56.0)  # by a tensor: a true division, not a product with 1 / 7
    e = torch.frexp(t).exponent - 1
    step = torch.exp2(e.clamp(min=-14).float() - 2)
    s = torch.round(t / step) * step
    byte = (s.half().view(torch.int16) >> 8).to(torch.uint8)
    byte = torch.where(fine, byte, 0x7F).to(torch.uint8)
    m = torch.floor(g.abs() / torch.where(s > 0, s, 1.0) + 0.5)
    n = (torch.where(g < 0, -m, m)).clamp(-8, 7) + 8
    n = torch.where(fine & (s > 0), n, 8.0).to(torch.uint8).reshape(*x.shape[:-1], x.shape[-1] // 2, 2)
    return n[..., 0] | (n[..., 1] << 4), byte.squeeze(-1)


def _values(codes, scales):
    """fp32 values of codes [..., D/2] with scale bytes [..., D/32]."""
    n = torch.stack((codes & 15, codes >> 4), dim=-1).float() - 8
    s = (scales.to(torch.int16) << 8).view(torch.float16).float()
    n = n.reshape(*codes.shape[:-1], scales.shape[-1], 32)
    return (n * s.unsqueeze(-1)).reshape(*codes.shape[:-1], codes.shape[-1] * 2)


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


def _plain_write(st, k, v):
    """Rows k, v [T, Hkv, D] into the cache; what it then holds of them, as fp32."""
    held = []
    for x, (codes, scales) in ((k, st["kc"]), (v, st["vc"])):
        c, s = _quantise(x)
        codes[st["seq"], :, st["pos"]] = c
        scales[st["seq"], :, st["pos"]] = s
        held.append(_values(c, s))
    return held


def _plain_attend(st, q):
    """q [T, Hq, D] (bf16 values) over the cache: causal softmax attention in fp32."""
    hkv, d, b = st["hkv"], st["d"], len(st["new"])
    g, lq, lk = st["hq"] // hkv, max(st["new"]), max(s + n for s, n in zip(st["start"], st["new"]))
    kf = _values(st["kc"][0][:, :, :lk], st["kc"][1][:, :, :lk])
    vf = _values(st["vc"][0][:, :, :lk], st["vc"][1][:, :, :lk])
    seen = torch.arange(lk, device=q.device) < st["end"].view(b, 1)  # rows that the sequence holds
    vf = torch.where(seen.view(b, 1, lk, 1), vf, 0.0)
    qp = torch.zeros(b, lq, hkv, g, d, device=q.device)
    qp[st["seq"], st["row"]] = q.float().view(-1, hkv, g, d)
    s = torch.matmul(qp.permute(0, 2, 3, 1, 4).reshape(b, hkv, g * lq, d), kf.transpose(-1, -2)) / math.sqrt(d)
    at = st["start_t"].view(b, 1) + torch.arange(lq, device=q.device)
    mask = torch.arange(lk, device=q.device) <= torch.minimum(at, st["end"].view(b, 1) - 1).unsqueeze(-1)
    s = s.view(b, hkv, g, lq, lk).masked_fill(~mask.view(b, 1, 1, lq, lk), -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).view(b, hkv, g * lq, lk)
    o = torch.matmul(p, vf).view(b, hkv, g, lq, d).permute(0, 3, 1, 2, 4)
    return o[st["seq"], st["row"]].reshape(-1, st["hq"], d).bfloat16()


# ------------------------------------------------------------------- the states
def _rows(gen, shape, gain):
    return (torch.randn(shape, generator=gen, device=DEV) * gain).bfloat16()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    hq, hkv, d, op = case["hq"], case["hkv"], case["d"], case["op"]
    start, new = _lens(case["start"]), _lens(case["new"])
    b, t, cap = len(new), sum(new), max(s + n for s, n in zip(start, new))
    # Keys and values of a layer differ in size from channel to channel.
    gk = torch.exp(0.4 * torch.randn(hkv, d, generator=gen, device=DEV))
    gv = torch.exp(0.4 * torch.randn(hkv, d, generator=gen, device=DEV))
    st = dict(op=op, hq=hq, hkv=hkv, d=d, start=start, new=new)
    st["k"], st["v"] = _rows(gen, (t, hkv, d), gk), _rows(gen, (t, hkv, d), gv)
    if op in ("decode", "prefill"):
        st["q"] = _rows(gen, (t, hq, d), 1.0)
        st["wq"] = (1 + 0.1 * torch.randn(d, generator=gen, device=DEV)).bfloat16()
        st["wk"] = (1 + 0.1 * torch.randn(d, generator=gen, device=DEV)).bfloat16()
    # The cache: random bytes where nothing has been written (scales that are NaN
    # among them), and rows of the same kind as the new ones where a sequence holds them.
    for name, gain in (("kc", gk), ("vc", gv)):
        codes = torch.randint(0, 256, (b, hkv, cap, d // 2), generator=gen, device=DEV, dtype=torch.uint8)
        scales = torch.randint(0, 128, (b, hkv, cap, d // 32), generator=gen, device=DEV, dtype=torch.uint8)
        for i in range(b):
            n = start[i] + (new[i] if op == "read" else 0)
            if n and op != "append":
                codes[i, :, :n], scales[i, :, :n] = _quantise(_rows(gen, (hkv, n, d), gain.unsqueeze(1)))
        st[name] = (codes, scales)
    dev = dict(device=DEV, dtype=torch.int64)
    st["seq"] = torch.repeat_interleave(torch.arange(b, **dev), torch.tensor(new, **dev))
    st["row"] = torch.cat([torch.arange(n, **dev) for n in new])
    st["start_t"] = torch.tensor(start, **dev)
    st["end"] = st["start_t"] + torch.tensor(new, **dev)
    st["pos"] = st["start_t"][st["seq"]] + st["row"]
    st["k_held"], st["v_held"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
    if op in ("decode", "prefill"):
        st["out"] = torch.empty_like(st["q"])
    if own:
        st["cache"] = _Cache(b, hq, hkv, d, cap)
        st["cache"].fill(st["kc"], st["vc"])
    return st


class _Cache:
    """The framework's 4-bit cache of one layer, freed with its state."""

    def __init__(self, b, hq, hkv, d, cap):
        from gqa_attention_preallocated_qa_gb300 import binding
        self.qa, self.shape = binding, (b, hkv, cap, d)
        self.handle = binding.qa_q4_cache_alloc(1, b, hq, hkv, d, cap, THETA, EPS)

    def fill(self, kc, vc):
        for view, own_bytes in zip(self.qa.q4_cache_tensors(self.handle, 0, *self.shape), (*kc, *vc)):
            view.copy_(own_bytes)

    def __del__(self):
        if getattr(self, "handle", None):
            self.qa.qa_q4_cache_free(self.handle)


def run(st):
    op = st["op"]
    if own:
        qa, cache = st["cache"].qa, st["cache"].handle
        if op == "append":
            qa.qa_q4_append(cache, 0, st["start"], st["new"], st["k"], st["v"], st["k_held"], st["v_held"])
            return {"k": st["k_held"], "v": st["v_held"]}
        if op == "read":
            qa.qa_q4_read(cache, 0, st["start"], st["new"], st["k_held"], st["v_held"])
            return {"k": st["k_held"], "v": st["v_held"]}
        if op == "decode":
            qa.qa_q4_decode_step(cache, 0, st["start"], st["q"], st["k"], st["v"], st["wq"], st["wk"], st["out"],
                                 st["k_held"], st["v_held"])
            return {"out": st["out"], "k": st["k_held"], "v": st["v_held"]}
        qa.qa_q4_prefill(cache, 0, st["start"], st["new"], st["q"], st["k"], st["v"], st["wq"], st["wk"], st["out"])
        # The appended values come back too.  (V only: a prompt's keys pass three
        # roundings before the quantiser, and of millions of them a few lie so near
        # a border that two right programs give neighbouring codes.)
        qa.qa_q4_read(cache, 0, st["start"], st["new"], None, st["v_held"])
        return {"out": st["out"], "v": st["v_held"]}
    if op == "append":
        k, v = _plain_write(st, st["k"], st["v"])
        return {"k": k.bfloat16(), "v": v.bfloat16()}
    if op == "read":
        k, v = (_values(c[st["seq"], :, st["pos"]], s[st["seq"], :, st["pos"]]).bfloat16() for c, s in (st["kc"], st["vc"]))
        return {"k": k, "v": v}
    k, v = _plain_write(st, _norm_rope(st["k"], st["wk"], st["pos"]), st["v"])
    out = _plain_attend(st, _norm_rope(st["q"], st["wq"], st["pos"]))
    if op == "decode":
        return {"out": out, "k": k.bfloat16(), "v": v.bfloat16()}
    return {"out": out, "v": v.bfloat16()}


# ------------------------------------------------------------------ in 64 bits
def _scale_table():
    """The value of each scale byte up to the largest (0x53), from its fields."""
    got = []
    for byte in range(0x54):
        e, m = byte >> 2, byte & 3
        got.append(m * 2.0 ** -16 if e == 0 else (4 + m) * 2.0 ** (e - 17))
    return torch.tensor(got, dtype=torch.float64, device=DEV)


def _exact_held(x):
    """The values that the cache holds for rows x, by search in the table of scales."""
    table = _scale_table()
    g = x.double().reshape(*x.shape[:-1], -1, 32)
    t = (g.abs().amax(-1, keepdim=True) / 7).contiguous()
    hi = torch.searchsorted(table, t).clamp(max=table.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = table[hi] - t, t - table[lo]
    s = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), table[hi], table[lo])
    quot = g / torch.where(s > 0, s, 1.0)
    n = (torch.sign(quot) * torch.floor(quot.abs() + 0.5)).clamp(-8, 7)
    return (n * s).reshape(x.shape)


def _exact_read(codes, scales, rows):
    table = torch.cat((_scale_table(), torch.full((256 - 0x54,), math.nan, dtype=torch.float64, device=DEV)))
    c = codes[:, :rows].long()
    n = torch.empty(*c.shape[:-1], c.shape[-1] * 2, dtype=torch.float64, device=DEV)
    n[..., 0::2], n[..., 1::2] = (c % 16).double(), (c // 16).double()
    return (n - 8) * table[scales[:, :rows].long()].repeat_interleave(32, -1)


def _exact_norm_rope(x, w, first):
    n, _, d = x.shape
    f = x.double()
    hat = (f / torch.sqrt((f * f).sum(-1, keepdim=True) / d + EPS)).bfloat16().double()
    y = (w.double() * hat).bfloat16().double()
    pos = torch.arange(first, first + n, device=DEV).double()
    i = torch.arange(d // 2, device=DEV).double()
    ang = pos[:, None] * torch.exp(-2.0 * i / d * math.log(THETA))[None]
    z = torch.complex(y[..., : d // 2], y[..., d // 2:]) * torch.polar(torch.ones_like(ang), ang)[:, None]
    return torch.cat((z.real, z.imag), -1).bfloat16().double()


def exact(case, seed):
    hq, hkv, d, op = case["hq"], case["hkv"], case["d"], case["op"]
    start, new = _lens(case["start"]), _lens(case["new"])
    st = prepare(case, seed)
    outs, ks, vs, at = [], [], [], 0
    for i, (s, n) in enumerate(zip(start, new)):
        k, v = st["k"][at:at + n], st["v"][at:at + n]
        if op == "read":
            ks.append(_exact_read(st["kc"][0][i], st["kc"][1][i], s + n)[:, s:].transpose(0, 1))
            vs.append(_exact_read(st["vc"][0][i], st["vc"][1][i], s + n)[:, s:].transpose(0, 1))
        elif op == "append":
            ks.append(_exact_held(k))
            vs.append(_exact_held(v))
        else:
            ks.append(_exact_held(_exact_norm_rope(k, st["wk"], s)))
            vs.append(_exact_held(v))
            q = _exact_norm_rope(st["q"][at:at + n], st["wq"], s)
            o = torch.empty(n, hq, d, dtype=torch.float64, device=DEV)
            kall = torch.cat((_exact_read(st["kc"][0][i], st["kc"][1][i], s), ks[-1].transpose(0, 1)), 1)
            vall = torch.cat((_exact_read(st["vc"][0][i], st["vc"][1][i], s), vs[-1].transpose(0, 1)), 1)
            unseen = torch.arange(s + n, device=DEV)[None] > torch.arange(s, s + n, device=DEV)[:, None]
            for h in range(hq):
                logit = q[:, h] @ kall[h // (hq // hkv)].T / math.sqrt(d)
                o[:, h] = torch.softmax(logit.masked_fill(unseen, -math.inf), -1) @ vall[h // (hq // hkv)]
            outs.append(o)
        at += n
    k, v = torch.cat(ks), torch.cat(vs)
    if op in ("append", "read"):
        return {"k": k, "v": v}
    out = torch.cat(outs)
    return {"out": out, "k": k, "v": v} if op == "decode" else {"out": out, "v": v}
