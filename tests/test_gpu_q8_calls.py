"""The 8-bit cache's calls on the GPU as callers make them: device positions, graphs,
streams, steps back, other caches beside it, refusals, and waits that run out."""
import numpy as np
import pytest
import torch

import q8_ref
from gpu_util import f64
from test_gpu_q8 import BLOCK, EPS, THETA, Cache, check_prefill, check_sparse, close, qa, rows  # noqa: F401

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def step(qa, c, lens, toks, w=(None, None), blocks=None, layer=0, stream=None):
    """A dense step, or a sparse one for blocks > 0; (out, list)."""
    q, k, v = toks
    out = torch.empty_like(q)
    if not blocks:
        qa.qa_q8_decode_step(c.h, layer, lens, q, k, v, *w, out, stream=stream)
        return out, None
    lists = torch.empty(len(lens), c.hkv, blocks, dtype=torch.int32, device="cuda")
    qa.qa_q8_sparse_step(c.h, layer, lens, blocks, q, k, v, *w, out, lists, stream=stream)
    return out, lists


# ------------------------------------------------------------------ device positions, graphs
@pytest.mark.parametrize("d", [64, 128])
def test_device_positions(qa, d):
    lens = [0, 63, 500, 1000]
    with Cache(qa, 4, 8, 2, d, 1100) as c:
        c.fill(lens, 3)
        q, k, v = c.tokens(4, 8)
        out = torch.empty_like(q)
        qa.qa_q8_decode_step_device_positions(c.h, 0, 4, ints(lens), q, k, v, None, None, out)
        c.ref.write(lens, [1] * 4, f64(k), f64(v))
        for b, pos in enumerate(lens):
            close(out[b:b + 1], *c.want(b, pos, q[b:b + 1].double()), what=f"position {pos}")
        lens = [n + 1 for n in lens]
        q, k, v = c.tokens(4, 18)
        lists = torch.empty(4, 2, 3, dtype=torch.int32, device="cuda")
        qa.qa_q8_sparse_step_device_positions(c.h, 0, 4, ints(lens), 3, q, k, v, None, None, out, lists)
        c.ref.write(lens, [1] * 4, f64(k), f64(v))
        for b, pos in enumerate(lens):
            close(out[b:b + 1], *c.want(b, pos, q[b:b + 1].double(), lists[b].cpu().numpy()), what=f"sparse, position {pos}")
        c.check_read([n + 1 for n in lens])


def test_device_position_out_of_range_leaves_its_sequence_alone(qa):
    lens = [100, 200, 64]
    with Cache(qa, 3, 8, 2, 128, 256) as c:
        c.fill(lens, 3)
        q, k, v = c.tokens(3, 8)
        for bad in (256, -1, 1 << 30):
            out = torch.full_like(q, 5.0)
            lists = torch.full((3, 2, 2), 77, dtype=torch.int32, device="cuda")
            qa.qa_q8_sparse_step_device_positions(c.h, 0, 3, ints([100, bad, 64]), 2, q, k, v, None, None, out, lists)
            assert qa.qa_q8_get_device_error(c.h)[0] == 8
            assert (out[1] == 5.0).all() and (lists[1] == -1).all() and (lists[0] >= -1).all() and (lists != 77).all()
            out.fill_(5.0)
            qa.qa_q8_decode_step_device_positions(c.h, 0, 3, ints([100, bad, 64]), q, k, v, None, None, out)
            assert qa.qa_q8_get_device_error(c.h)[0] == 8
            assert qa.qa_q8_get_device_error(c.h) == (0, 0)
            assert (out[1] == 5.0).all()
        c.ref.write(lens, [1, 0, 1], f64(k)[[0, 2]], f64(v)[[0, 2]])
        for b in (0, 2):
            close(out[b:b + 1], *c.want(b, lens[b], q[b:b + 1].double()))
        c.check_read([101, 200, 65])


@pytest.mark.parametrize("blocks", [0, 2])
def test_steps_in_a_graph_advance_through_a_block(qa, blocks):
    """Three layers, positions advanced inside the graph; the same eagerly, bit for bit."""
    lens, layers, steps = [50, 190, 320], 3, 20
    outs = []
    for graphed in (True, False):
        with Cache(qa, 3, 8, 2, 128, 400, layers=layers) as c:
            for layer in range(layers):
                k, v = rows(layer, sum(lens), 2, 128), rows(9 + layer, sum(lens), 2, 128)
                qa.qa_q8_append(c.h, layer, [0] * 3, lens, k, v)
            pos = ints(lens)
            q, k, v = c.tokens(3, 40)
            out = torch.empty(layers, *q.shape, dtype=torch.bfloat16, device="cuda")
            lists = torch.empty(layers, 3, 2, max(1, blocks), dtype=torch.int32, device="cuda")

            def one():
                for layer in range(layers):
                    if blocks:
                        qa.qa_q8_sparse_step_device_positions(c.h, layer, 3, pos, blocks, q, k, v, c.wq, c.wk, out[layer], lists[layer])
                    else:
                        qa.qa_q8_decode_step_device_positions(c.h, layer, 3, pos, q, k, v, c.wq, c.wk, out[layer])
                pos.add_(1)

            one()
            if graphed:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    one()
            got = []
            for i in range(steps):
                q.copy_(rows(100 + i, *q.shape))
                k.copy_(rows(200 + i, *k.shape))
                v.copy_(rows(300 + i, *v.shape))
                graph.replay() if graphed else one()
                got.append((out.clone(), lists.clone()))
            held = [torch.empty(3 * 50, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            qa.qa_q8_read(c.h, 1, [20, 160, 290], [50] * 3, *held)
            outs.append((got, held))
            assert qa.qa_q8_get_device_error(c.h)[0] == 0
    for a, b in zip(outs[0][0], outs[1][0]):
        assert torch.equal(a[0], b[0]) and (not blocks or torch.equal(a[1], b[1]))
    assert all(torch.equal(a, b) for a, b in zip(outs[0][1], outs[1][1]))


def test_rows_and_host_positions_in_a_graph(qa):
    with Cache(qa, 2, 8, 2, 128, 300) as c:
        c.fill([100, 63], 3)
        q, k, v = c.tokens(2, 8)
        kr, vr = rows(5, 40, 2, 128), rows(6, 40, 2, 128)
        out, ko, vo = torch.empty_like(q), torch.empty_like(kr), torch.empty_like(vr)

        def calls():
            qa.qa_q8_append(c.h, 0, [100, 63], [30, 10], kr, vr)
            qa.qa_q8_decode_step(c.h, 0, [130, 73], q, k, v, None, None, out)
            qa.qa_q8_read(c.h, 0, [100, 63], [30, 10], ko, vo)
        calls()
        want = [x.clone() for x in (out, ko, vo)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            calls()
        for _ in range(3):
            for x in (out, ko, vo):
                x.zero_()
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(want, (out, ko, vo)))


# ------------------------------------------------------------------ order of calls
@pytest.mark.parametrize("d", [64, 128])
def test_calls_in_a_row_are_as_calls_one_by_one(qa, d):
    """Steps of several layers and of one, rows, reads and sparse steps without a
    synchronisation between them, against the same with one: the same bits."""
    got = []
    for apart in (True, False):
        with Cache(qa, 3, 16, 2, d, 700, layers=4) as c:
            lens = [500, 63, 127]
            for layer in range(4):
                qa.qa_q8_append(c.h, layer, [0] * 3, lens, rows(layer, sum(lens), 2, d), rows(9 + layer, sum(lens), 2, d))
            toks = [c.tokens(3, 100 + 3 * i) for i in range(40)]
            torch.cuda.synchronize()
            seen = []
            for i in range(40):
                layer = [0, 1, 2, 3, 0, 0, 1, 1][i % 8]
                here = [n + i for n in lens]  # (the layers' other rows are whatever they were)
                out, lists = step(qa, c, here, toks[i], blocks=[0, 0, 2, 0, 0, 3][i % 6], layer=layer)
                seen += [out] if lists is None else [out, lists]
                if apart:
                    torch.cuda.synchronize()
                if i % 5 == 4:
                    kv = [torch.empty(3 * 8, 2, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
                    qa.qa_q8_read(c.h, layer, [n - 7 for n in here], [8] * 3, *kv)
                    seen += kv
                if i % 7 == 6:
                    qa.qa_q8_append(c.h, layer, here, [2, 0, 1], rows(i, 3, 2, d), rows(i + 1, 3, 2, d))
                if apart:
                    torch.cuda.synchronize()
            torch.cuda.synchronize()
            got.append(seen)
            assert qa.qa_q8_get_device_error(c.h)[0] == 0
    for i, (a, b) in enumerate(zip(*got)):
        assert torch.equal(a, b), i


def test_steps_beside_the_other_caches_on_one_stream(qa):
    geo = (1, 2, 16, 2, 128, 400)
    lens, got = [300, 65], []
    for apart in (True, False):
        bf16, q4 = qa.qa_cache_alloc(*geo, THETA, EPS), qa.qa_q4_cache_alloc(*geo, THETA, EPS)
        with Cache(qa, 2, 16, 2, 128, 400) as c:
            try:
                k, v = rows(1, sum(lens), 2, 128), rows(2, sum(lens), 2, 128)
                kt, vt, _ = qa.cache_tensors(bf16, 0, 2, 2, 400, 128)
                for b, (at, n) in enumerate(((0, 300), (300, 65))):
                    kt[b, :, :n], vt[b, :, :n] = k[at:at + n].transpose(0, 1), v[at:at + n].transpose(0, 1)
                qa.qa_cache_set_lengths(bf16, 0, lens)
                qa.qa_q4_append(q4, 0, [0, 0], lens, k, v)
                qa.qa_q8_append(c.h, 0, [0, 0], lens, k, v)
                toks = [c.tokens(2, 100 + 3 * i) for i in range(30)]
                torch.cuda.synchronize()
                seen = []
                for i, (q, kk, vv) in enumerate(toks):
                    here = [n + i for n in lens]
                    for which in (0, 1, 2) if i % 2 else (2, 0, 2, 1):
                        out = torch.empty_like(q)
                        if which == 0:
                            qa.qa_decode_step(bf16, 0, 2, q, kk, vv, c.wq, c.wk, out)
                        elif which == 1:
                            qa.qa_q4_decode_step(q4, 0, here, q, kk, vv, c.wq, c.wk, out)
                        else:
                            qa.qa_q8_decode_step(c.h, 0, here, q, kk, vv, c.wq, c.wk, out)
                        seen.append(out)
                        if apart:
                            torch.cuda.synchronize()
                torch.cuda.synchronize()
                got.append(seen)
            finally:
                qa.qa_cache_free(bf16)
                qa.qa_q4_cache_free(q4)
    for i, (a, b) in enumerate(zip(*got)):
        close(b, a.double(), 0 * a.double().abs() + 8.0 * 2.0 ** -8, 0 * a.double(), what=f"call {i}")


def test_a_step_is_the_same_every_time(qa):
    lens = [900, 64, 333]
    with Cache(qa, 3, 32, 4, 64, 1000) as c:
        c.fill(lens, 3)
        toks = c.tokens(3, 8)
        first = step(qa, c, lens, toks)[0]
        sparse, lists = step(qa, c, lens, toks, blocks=4)
        for _ in range(20):
            assert torch.equal(step(qa, c, lens, toks)[0], first)
            again = step(qa, c, lens, toks, blocks=4)
            assert torch.equal(again[0], sparse) and torch.equal(again[1], lists)


def test_on_another_stream(qa):
    lens, side = [200, 130], torch.cuda.Stream()
    with Cache(qa, 2, 8, 2, 128, 400) as c:
        c.fill(lens, 3)
        toks = c.tokens(2, 8)
        torch.cuda.synchronize()
        out, _ = step(qa, c, lens, toks, stream=side)
        side.synchronize()
        c.ref.write(lens, [1, 1], f64(toks[1]), f64(toks[2]))
        for b, pos in enumerate(lens):
            close(out[b:b + 1], *c.want(b, pos, toks[0][b:b + 1].double()))


def test_two_threads_on_caches_of_their_own(qa):
    """Each on its own stream: steps of both kinds, rows and a prompt, at once."""
    import threading

    def work(seed, stream, got):
        lens = [300, 129]
        with torch.cuda.stream(stream), Cache(qa, 2, 8, 2, 128, 700) as c:
            q, k, v = c.tokens(sum(lens), seed)
            out = torch.empty_like(q)
            qa.qa_q8_prefill(c.h, 0, [0, 0], lens, q, k, v, c.wq, c.wk, out, stream)
            got.append(out)
            for i in range(20):
                o, lists = step(qa, c, [n + i for n in lens], c.tokens(2, seed + i), blocks=2 if i % 2 else 0, stream=stream)
                got += [o] + ([lists] if i % 2 else [])
            kv = torch.empty(2 * 20, 2, 128, device="cuda", dtype=torch.bfloat16)
            qa.qa_q8_read(c.h, 0, lens, [20, 20], kv, None, stream)
            got.append(kv)
            stream.synchronize()

    alone = [[], []]
    for i in range(2):
        work(100 * i, torch.cuda.Stream(), alone[i])
    for _ in range(3):
        both = [[], []]
        threads = [threading.Thread(target=work, args=(100 * i, torch.cuda.Stream(), both[i])) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join(120)
        for a, b in zip(alone, both):
            assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_prefill_on_two_streams_shares_the_workspace(qa):
    streams = [torch.cuda.Stream() for _ in range(2)]
    with Cache(qa, 1, 8, 2, 128, 600, layers=2) as c, Cache(qa, 1, 8, 2, 128, 600) as one:
        toks = [c.tokens(500, 10 + 3 * i) for i in range(2)]
        want = []
        for q, k, v in toks:
            out = torch.empty_like(q)
            qa.qa_q8_prefill(one.h, 0, [0], [500], q, k, v, c.wq, c.wk, out)
            want.append(out)
        torch.cuda.synchronize()
        for _ in range(5):
            outs = []
            for layer, (s, (q, k, v)) in enumerate(zip(streams, toks)):
                out = torch.empty_like(q)
                qa.qa_q8_prefill(c.h, layer, [0], [500], q, k, v, c.wq, c.wk, out, s)
                outs.append(out)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want))


# ------------------------------------------------------------------ positions again
@pytest.mark.parametrize("d", [64, 128])
def test_a_dropped_token_is_written_again(qa, d):
    """In the block being filled and, over its border, in the one before: as if the
    dropped tokens had never been."""
    for lens, back in (([70, 90], 5), ([66, 130], 5), ([64, 128], 1), ([65, 129], 30)):
        with Cache(qa, 2, 4, 2, d, 256) as c:
            for pos in range(0, max(lens)):
                n = [int(pos < x) for x in lens]
                q, k, v = c.tokens(2, 3 * pos)
                if all(n):
                    step(qa, c, [pos, pos], (q, k, v))
                    c.ref.write([pos, pos], [1, 1], f64(k), f64(v))
                else:  # the longer one alone, by rows
                    k, v = k[:1].contiguous(), v[:1].contiguous()
                    c.append([0, pos], [0, 1], k, v)
            here = [n - back for n in lens]
            q, k, v = c.tokens(2, 999)
            out, _ = step(qa, c, here, (q, k, v))
            c.ref.write(here, [1, 1], f64(k), f64(v))
            for b, pos in enumerate(here):
                close(out[b:b + 1], *c.want(b, pos, q[b:b + 1].double()), what=f"{lens[b]} back by {back}")
            here = [n + 1 for n in here]
            k, v = rows(5, 140, 2, d), rows(6, 140, 2, d)
            c.append(here, [70, 70], k, v)
            c.check_read([n + 70 for n in here])


@pytest.mark.parametrize("by", ["step", "rows", "prefill"])
def test_a_step_back_by_many_blocks_takes_the_held_values(qa, by):
    d, back = 128, 100
    with Cache(qa, 1, 4, 2, d, 700) as c:
        c.fill([640], 3)
        # rows 64..99 of the block come back as the cache held them
        for i in range(2):
            held = q8_ref.bf16(q8_ref.values(c.ref.n[i, 0, :, 1], c.ref.s[i, 0, :, 1]))
            c.ref.came[i, 0, :, BLOCK:back] = held[:, :back - BLOCK]
        if by == "prefill":
            check_prefill(qa, c, [back], [30], 8)
            c.check_read([back + 30])
            return
        q, k, v = c.tokens(1, 8)
        if by == "step":
            out, _ = step(qa, c, [back], (q, k, v))
            c.ref.write([back], [1], f64(k), f64(v))
            close(out, *c.want(0, back, q.double()))
        else:
            c.append([back], [1], k, v)
        c.check_read([back + 1])
        k, v = rows(5, 60, 2, d), rows(6, 60, 2, d)
        c.append([back + 1], [60], k, v)
        c.check_read([back + 61])


def test_rows_behind_the_position_are_not_seen(qa):
    """NaN in every row from the position on, in complete blocks and in the one being filled."""
    d = 128
    with Cache(qa, 2, 8, 2, d, 900) as c:
        lens = [300, 64]
        c.fill(lens, 3)
        bad = torch.full((900 - 300 + 900 - 64, 2, d), float("nan"), device="cuda", dtype=torch.bfloat16)
        qa.qa_q8_append(c.h, 0, lens, [600, 836], bad, bad)
        kept = c.ref.came.copy()
        for i in range(2):  # rows 256..299 of sequence 0: complete with the NaN, and kept as they came
            assert np.isfinite(kept[i, 0, :, 256:300]).all()
        for blocks in (0, 3):
            q, k, v = c.tokens(2, 8)
            out, lists = step(qa, c, lens, (q, k, v), blocks=blocks)
            assert torch.isfinite(out).all()
            c.ref.write(lens, [1, 1], f64(k), f64(v))
            for b, pos in enumerate(lens):
                close(out[b:b + 1], *c.want(b, pos, q[b:b + 1].double(), lists[b].cpu().numpy() if blocks else None))
            lens = [n + 1 for n in lens]
        lens = check_prefill(qa, c, lens, [40, 70], 20)
        c.check_read(lens)


def test_values_that_are_not_finite_reach_their_heads_alone(qa):
    lens = [300]
    with Cache(qa, 1, 8, 2, 128, 400) as c:
        k, v = rows(1, 300, 2, 128), rows(2, 300, 2, 128)
        k[17, 1, 5] = float("inf")
        c.append([0], [300], k, v)
        out, _ = step(qa, c, lens, c.tokens(1, 8))
        assert torch.isfinite(out[0, :4]).all() and torch.isnan(out[0, 4:]).all()
    with Cache(qa, 1, 8, 2, 128, 400) as c:
        k, v = rows(1, 300, 2, 128), rows(2, 300, 2, 128)
        v[299, 0, 9] = float("nan")  # in the block being filled: one dimension
        c.append([0], [300], k, v)
        out, _ = step(qa, c, lens, c.tokens(1, 8))
        bad = torch.isnan(out[0])
        assert bad[:4, 9].all() and bad.sum() == 4


# ------------------------------------------------------------------ sizes
def test_more_sequences_than_a_launch(qa):
    n = 70
    with Cache(qa, n, 2, 1, 64, 200) as c:
        lens = [(37 * i) % 190 for i in range(n)]
        c.fill(lens, 3)
        c.check_read(lens)
        toks = c.tokens(n, 8)
        out, lists = step(qa, c, lens, toks, blocks=2)
        assert qa.qa_q8_stats(c.h) == {"write": 2, "read": 2, "prefill_attn": 0, "decode": 0, "sparse": 2}
        c.ref.write(lens, [1] * n, f64(toks[1]), f64(toks[2]))
        for b, pos in enumerate(lens):
            close(out[b:b + 1], *c.want(b, pos, toks[0][b:b + 1].double(), lists[b].cpu().numpy()), what=f"sequence {b}")
        c.check_read([x + 1 for x in lens])


def test_sequences_behind_the_batch_are_left_alone(qa):
    with Cache(qa, 3, 4, 2, 64, 200) as c:
        c.fill([100, 64, 130], 3)
        k, v = rows(5, 30, 2, 64), rows(6, 30, 2, 64)
        c.append([100], [30], k, v)
        step(qa, c, [130], c.tokens(1, 8))
        q, k, v = c.tokens(5, 9)
        qa.qa_q8_prefill(c.h, 0, [131], [5], q, k, v, c.wq, c.wk, torch.empty_like(q))
        for b, n in ((1, 64), (2, 130)):
            ko, vo = (torch.empty(n, 2, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
            qa.qa_q8_read(c.h, 0, [0] * (b + 1), [0] * b + [n], ko, vo)
            np.testing.assert_array_equal(f64(ko), c.ref.read(0, b, 0, n, n))
            np.testing.assert_array_equal(f64(vo), c.ref.read(1, b, 0, n, n))


def test_offsets_past_32_bits(qa):
    """The codes of the layer's last sequence lie 2^31 bytes and more behind its first's."""
    cap, hkv = 1 << 18, 8
    with Cache(qa, 1, 8, hkv, 128, 64) as c:  # (its reference alone)
        h = qa.qa_q8_cache_alloc(1, 5, 8, hkv, 128, cap, THETA, EPS)
        try:
            assert qa.qa_q8_memory_info(h)[0] > 5 << 29
            k, v = rows(1, 700, hkv, 128), rows(2, 700, hkv, 128)
            ref = q8_ref.Rows(1, hkv, 128, 1024)
            ref.write([0], [700], f64(k), f64(v))
            qa.qa_q8_append(h, 0, [0] * 5, [0, 0, 0, 0, 700], k, v)
            ko, vo = torch.empty_like(k), torch.empty_like(v)
            qa.qa_q8_read(h, 0, [0] * 5, [0, 0, 0, 0, 700], ko, vo)
            np.testing.assert_array_equal(f64(ko), ref.read(0, 0, 0, 700, 700))
            q, kn, vn = rows(5, 5, 8, 128), rows(6, 5, hkv, 128), rows(7, 5, hkv, 128)
            out, lists = torch.empty_like(q), torch.empty(5, hkv, 3, dtype=torch.int32, device="cuda")
            lens = [0, 0, 0, 0, 700]
            for blocks in (0, 3):
                if blocks:
                    qa.qa_q8_sparse_step(h, 0, lens, 3, q, kn, vn, None, None, out, lists)
                else:
                    qa.qa_q8_decode_step(h, 0, lens, q, kn, vn, None, None, out)
                for g in range(hkv):
                    kk, vv = (torch.from_numpy(np.concatenate((ref.held(i, 0, 700, lists[4].cpu().numpy() if blocks else None)[g],
                                                               f64(x)[4:, g]))).cuda()[None]
                              for i, x in enumerate((kn, vn)))
                    close(out[4:, g:g + 1], *q8_ref.attend(q[4:, g:g + 1].double(), kk, vv, kk.shape[1] - 1))
                assert torch.equal(out[:4], vn[:4])  # alone with themselves
        finally:
            qa.qa_q8_cache_free(h)


def test_memory(qa):
    """The cache's size, and that only a first prefill allocates."""
    with Cache(qa, 4, 8, 2, 128, 1000) as c:
        held, scratch = qa.qa_q8_memory_info(c.h)
        blocks = 16 * 8
        assert held == blocks * (2 * 64 * 128 + 8 + 2 * 128) + 8 * (2 * 2 * 64 * 128 * 2 + 16)
        assert scratch >= 2 * 4 * 2 * 1000 * 128 * 2
        lens = [500, 63, 1, 900]

        def calls(prefill):
            c.append([0] * 4, lens, rows(1, sum(lens), 2, 128), rows(2, sum(lens), 2, 128))
            step(qa, c, lens, c.tokens(4, 5))
            step(qa, c, lens, c.tokens(4, 5), blocks=3)
            if prefill:
                q, k, v = c.tokens(40, 9)
                qa.qa_q8_prefill(c.h, 0, [0], [40], q, k, v, c.wq, c.wk, torch.empty_like(q))
            torch.cuda.synchronize()
        for prefill in (False, True):
            calls(prefill)
            before = torch.cuda.mem_get_info()[0] + torch.cuda.memory_reserved()
            for _ in range(3):
                calls(prefill)
            assert torch.cuda.mem_get_info()[0] + torch.cuda.memory_reserved() == before


# ------------------------------------------------------------------ refusals, failures
def test_refusals_change_nothing(qa):
    with Cache(qa, 2, 8, 2, 128, 128) as c:
        c.fill([70, 20], 5)
        q, k, v = c.tokens(2, 6)
        out = torch.full_like(q, 3.0)
        lists = torch.full((2, 2, 2), 3, dtype=torch.int32, device="cuda")
        w = (c.wq, c.wk)

        def refused(status, fn, *args):
            with pytest.raises(qa.QaError) as e:
                fn(c.h, *args)
            assert e.value.status == status, args

        odd = q.view(-1)[1:]
        for layer in (-1, 1):
            refused(1, qa.qa_q8_append, layer, [0], [1], k, v)
            refused(1, qa.qa_q8_read, layer, [0], [1], k, v)
            refused(1, qa.qa_q8_prefill, layer, [0], [1], q, k, v, *w, out)
            refused(1, qa.qa_q8_decode_step, layer, [0], q, k, v, *w, out)
        refused(1, qa.qa_q8_append, 0, [0, 0, 0], [1, 1, 1], k, v)      # more than max_batch
        refused(1, qa.qa_q8_append, 0, [], [], k, v)
        refused(1, qa.qa_q8_append, 0, [-1], [1], k, v)
        refused(1, qa.qa_q8_append, 0, [0], [-1], k, v)
        refused(4, qa.qa_q8_append, 0, [127, 0], [2, 1], k, v)
        refused(4, qa.qa_q8_append, 0, [2 ** 31 - 1], [2 ** 31 - 1], k, v)
        refused(1, qa.qa_q8_append, 0, [0], [1], None, v)
        refused(3, qa.qa_q8_append, 0, [0], [1], odd, v)
        refused(4, qa.qa_q8_read, 0, [128], [1], k, v)
        refused(1, qa.qa_q8_read, 0, [0], [1], None, None)
        refused(3, qa.qa_q8_read, 0, [0], [1], k, odd)
        refused(1, qa.qa_q8_read, 0, [0], [1], k, k)
        refused(4, qa.qa_q8_prefill, 0, [127], [2], q, k, v, *w, out)
        refused(1, qa.qa_q8_prefill, 0, [0], [2], q, k, v, None, c.wk, out)
        refused(1, qa.qa_q8_prefill, 0, [0], [2], q, k, v, *w, q)
        refused(3, qa.qa_q8_prefill, 0, [0], [2], q, k, v, *w, odd)
        for n in (None, 2):
            fn = qa.qa_q8_sparse_step if n else qa.qa_q8_decode_step
            dev = qa.qa_q8_sparse_step_device_positions if n else qa.qa_q8_decode_step_device_positions
            head = (lambda p: (0, p, n)) if n else (lambda p: (0, p))
            last = (lists,) if n else ()
            refused(4, fn, *head([128, 0]), q, k, v, *w, out, *last)
            refused(1, fn, *head([0, -1]), q, k, v, *w, out, *last)
            refused(1, fn, *head([0]), q, k, v, *w, None, *last)
            refused(1, fn, *head([0]), q, k, v, c.wq, None, out, *last)
            refused(1, fn, *head([0]), q, k, v, *w, out, *last, k.clone(), None)
            refused(1, fn, *head([0]), q, k, v, *w, q, *last)
            refused(1, fn, *head([0]), q, k, v, *w, out, *last, k, v)
            refused(1, fn, *head([0, 0]), q, k, v, *w, out, *last, out, k.clone())
            refused(3, fn, *head([0]), q, odd, v, *w, out, *last)
            refused(1, dev, 0, 1, None, *((n,) if n else ()), q, k, v, *w, out, *last)
        for n in (0, -1, 3):
            refused(1, qa.qa_q8_sparse_step, 0, [0], n, q, k, v, *w, out, lists)
        refused(1, qa.qa_q8_sparse_step, 0, [0], 2, q, k, v, *w, out, None)
        refused(3, qa.qa_q8_sparse_step, 0, [0], 2, q, k, v, *w, out, lists.data_ptr() + 2)
        refused(1, qa.qa_q8_sparse_step, 0, [0, 0], 2, q, k, v, *w, out, out)
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.stream(side):
            graph.capture_begin()
            try:
                refused(5, qa.qa_q8_prefill, 0, [20], [2], q, k, v, *w, out, side)
            finally:
                graph.capture_end()
        torch.cuda.synchronize()
        assert (out == 3.0).all() and (lists == 3).all()
        c.check_read([70, 20])
        qa.qa_q8_append(c.h, 0, [0, 128], [0, 0], None, None)  # no rows: nothing to do
        assert qa.qa_q8_stats(c.h) == {"write": 1, "read": 1, "prefill_attn": 0, "decode": 0, "sparse": 0}


@pytest.mark.parametrize("blocks", [0, 4, 8])
@pytest.mark.parametrize("lens", [[700, 1100], [1100, 90, 0, 7]])
def test_a_wait_that_runs_out_is_reported_and_the_cache_stays_usable(qa, lens, blocks):
    # Four blocks (and 17 / 32 for their choice) are one CTA's: it waits for nobody.
    several = blocks != 4
    with Cache(qa, len(lens), 32, 8, 128, 1200) as c:
        c.fill(lens, 3)
        toks = c.tokens(len(lens), 8)
        assert qa.qa_q8_get_device_error(c.h) == (0, 0)
        qa.qa_debug_arm_wait_timeout(2, 20000)  # the next decode launch: 20 ms
        try:
            step(qa, c, lens, toks, blocks=blocks)
            st, word = qa.qa_q8_get_device_error(c.h)
            assert (st == 7 and word & 0xff == 1 and word >> 8 & 0xff == 7) if several else (st, word) == (0, 0)
        finally:
            qa.qa_debug_arm_wait_timeout(-1, 0)
        out, lists = step(qa, c, lens, toks, blocks=blocks)
        assert qa.qa_q8_get_device_error(c.h) == (0, 0)
        c.ref.write(lens, [1] * len(lens), f64(toks[1]), f64(toks[2]))
        for b, pos in enumerate(lens):
            close(out[b:b + 1], *c.want(b, pos, toks[0][b:b + 1].double(), lists[b].cpu().numpy() if blocks else None))


def test_a_prefill_whose_wait_runs_out(qa):
    with Cache(qa, 2, 8, 2, 128, 700) as c:
        c.fill([300, 0], 3)
        q, k, v = c.tokens(200, 8)
        out = torch.empty_like(q)
        qa.qa_debug_arm_wait_timeout(1, 20000)
        try:
            qa.qa_q8_prefill(c.h, 0, [300, 0], [100, 100], q, k, v, c.wq, c.wk, out)
            st, word = qa.qa_q8_get_device_error(c.h)
            assert st == 7 and word & 0xff == 1
        finally:
            qa.qa_debug_arm_wait_timeout(-1, 0)
        check_prefill(qa, c, [300, 0], [100, 100], 8)
        assert qa.qa_q8_get_device_error(c.h) == (0, 0)


@pytest.mark.parametrize("blocks", [0, 8])
def test_who_gave_up_waiting_stays_for_what_is_late(qa, blocks):
    """A thread block whose wait ran out leaves after a second limit, in which what the others
    of its cluster may still send it finds it there."""
    lens, limit_us = [700, 1100], 20000
    with Cache(qa, len(lens), 32, 8, 128, 1200) as c:
        c.fill(lens, 3)
        toks = c.tokens(len(lens), 8)
        step(qa, c, lens, toks, blocks=blocks)
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        qa.qa_debug_arm_wait_timeout(2, limit_us)
        try:
            begin.record()
            step(qa, c, lens, toks, blocks=blocks)
            end.record()
            st, word = qa.qa_q8_get_device_error(c.h)
            assert st == 7 and word & 0xff == 1 and word >> 8 & 0xff == 7
        finally:
            qa.qa_debug_arm_wait_timeout(-1, 0)
        assert begin.elapsed_time(end) >= 2 * limit_us * 1e-3
