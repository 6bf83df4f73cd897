"""Steps on two streams that wait for each other's events, as they run and in a graph:
the bits of the same calls one by one.  Each step depends on rows that the one before it
on the other stream writes."""
import pytest
import torch

pytestmark = pytest.mark.gpu

THETA, EPS = 1e6, 1e-6
HQ, HKV, D, LAYERS = 8, 2, 128, 2


@pytest.fixture(scope="module")
def qa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gqa_attention_preallocated_qa_gb300 import _build
    _build.build()
    from gqa_attention_preallocated_qa_gb300 import binding
    return binding


def rows(seed, *shape):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").bfloat16()


class Bf16:
    """Steps with device lengths (their split plan is the same on any stream)."""

    def __init__(self, qa, length, cap):
        self.qa, self.len = qa, length
        self.h = qa.qa_cache_alloc(LAYERS, 1, HQ, HKV, D, cap, THETA, EPS)
        for layer in range(LAYERS):
            k, v, _ = qa.cache_tensors(self.h, layer, 1, HKV, cap, D)
            k[0, :, :length] = rows(layer, HKV, length, D)
            v[0, :, :length] = rows(9 + layer, HKV, length, D)
            qa.qa_cache_set_lengths(self.h, layer, [length])

    def step(self, layer, pos, toks, w, out, stream):
        self.qa.qa_decode_step_device_lengths(self.h, layer, 1, *toks, *w, out, stream)

    def error(self):
        return self.qa.qa_get_device_error(self.h)

    def close(self):
        self.qa.qa_cache_free(self.h)


class Q4:
    name = "q4"

    def __init__(self, qa, length, cap):
        self.qa = qa
        self.h = self.fn("cache_alloc")(LAYERS, 1, HQ, HKV, D, cap, THETA, EPS)
        for layer in range(LAYERS):
            self.fn("append")(self.h, layer, [0], [length], rows(layer, length, HKV, D), rows(9 + layer, length, HKV, D))

    def fn(self, what):
        return getattr(self.qa, f"qa_{self.name}_{what}")

    def step(self, layer, pos, toks, w, out, stream):
        self.fn("decode_step")(self.h, layer, [pos], *toks, *w, out, stream=stream)

    def error(self):
        return self.fn("get_device_error")(self.h)

    def close(self):
        self.fn("cache_free")(self.h)


class Q8(Q4):
    name = "q8"


class Q8Sparse(Q8):
    def step(self, layer, pos, toks, w, out, stream):
        self.lists = getattr(self, "lists", [])  # (kept: the streams write them later)
        self.lists.append(torch.empty(1, HKV, 4, dtype=torch.int32, device="cuda"))
        self.qa.qa_q8_sparse_step(self.h, layer, [pos], 4, *toks, *w, out, self.lists[-1], stream=stream)


class Q8Rows(Q8):
    """Every other step is rows alone."""

    def step(self, layer, pos, toks, w, out, stream):
        if pos % 2:
            super().step(layer, pos, toks, w, out, stream)
        else:
            self.qa.qa_q8_append(self.h, layer, [pos], [1], toks[1], toks[2], stream)


# (stream, layer): "wait" has the stream wait for all that the other one has so far
FORKED = [(0, 0), (1, "wait"), (1, 0), (0, 1), (1, 0), (0, "wait"), (0, 0), (0, 1), (0, 0), (1, "wait"), (1, 1), (1, 0), (1, 1),
          (0, "wait"), (0, 1), (0, 0)]


@pytest.mark.parametrize("length", [500, 6000])
@pytest.mark.parametrize("cache", [Bf16, Q4, Q8, Q8Sparse, Q8Rows])
def test_steps_of_streams_that_wait_for_each_other(qa, cache, length):
    cap = length + 40
    w = (1 + 0.1 * rows(1, D), 1 + 0.1 * rows(2, D))
    toks = [(rows(50 + 3 * i, 1, HQ, D), rows(51 + 3 * i, 1, HKV, D), rows(52 + 3 * i, 1, HKV, D)) for i in range(len(FORKED))]

    def run(c, outs, streams, apart):
        at = [length] * LAYERS
        for i, (s, layer) in enumerate(FORKED):
            if layer == "wait":
                event = torch.cuda.Event()
                event.record(streams[1 - s])
                streams[s].wait_event(event)
                continue
            c.step(layer, at[layer], toks[i], w, outs[i], streams[s])
            at[layer] += 1
            if apart:
                torch.cuda.synchronize()

    got = []
    for how in ("apart", "run", "graph"):
        c = cache(qa, length, cap)
        try:
            outs = torch.zeros(len(FORKED), 1, HQ, D, device="cuda", dtype=torch.bfloat16)
            streams = [torch.cuda.Stream(), torch.cuda.Stream()]
            torch.cuda.synchronize()
            if how == "graph":
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=streams[0]):
                    run(c, outs, streams, False)
                torch.cuda.synchronize()
                graph.replay()
            else:
                run(c, outs, streams, how == "apart")
            torch.cuda.synchronize()
            assert c.error()[0] == 0
            got.append(outs.clone())
        finally:
            c.close()
    for how, x in zip(("run", "graph"), got[1:]):
        for i in range(len(FORKED)):
            assert torch.equal(got[0][i], x[i]), f"{how}: call {i}"


@pytest.mark.parametrize("cache", [Bf16, Q4, Q8, Q8Sparse])
def test_a_step_behind_a_graph(qa, cache):
    """A graph's last kernel lets its successors start early; the step that follows the
    graph's launch depends on the rows that it writes."""
    length = 6000
    w = (1 + 0.1 * rows(1, D), 1 + 0.1 * rows(2, D))
    toks = [(rows(50 + 3 * i, 1, HQ, D), rows(51 + 3 * i, 1, HKV, D), rows(52 + 3 * i, 1, HKV, D)) for i in range(4)]
    got = []
    for apart in (True, False):
        c, side = cache(qa, length, length + 10), torch.cuda.Stream()
        try:
            outs = torch.zeros(4, 1, HQ, D, device="cuda", dtype=torch.bfloat16)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
                c.step(1, length, toks[0], w, outs[0], torch.cuda.current_stream())
                c.step(0, length, toks[1], w, outs[1], torch.cuda.current_stream())
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                graph.replay()
                if apart:
                    torch.cuda.synchronize()
                c.step(0, length + 1, toks[2], w, outs[2], side)
                c.step(1, length + 1, toks[3], w, outs[3], side)
            torch.cuda.synchronize()
            assert c.error()[0] == 0
            got.append(outs.clone())
        finally:
            c.close()
    assert torch.equal(*got)
