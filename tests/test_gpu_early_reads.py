"""Steps behind a kernel of other code that signals before it has stored their inputs, with
early reads off (qa_set_early_reads): the bits of the same steps with their inputs at rest."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from test_gpu_forks import D, HKV, HQ, Bf16, Q4, Q8, Q8Sparse, qa, rows  # noqa: F401

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def producer(qa, tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    lib = str(tmp_path_factory.mktemp("producer") / "early_producer.so")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-shared", "-Xcompiler", "-fPIC",
                    os.path.join(HERE, "native", "early_producer.cu"), "-o", lib], check=True)
    fn = ctypes.CDLL(lib).launch_early_producer
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_void_p]
    return fn


@pytest.mark.parametrize("graphed", [False, True])
@pytest.mark.parametrize("cache", [Bf16, Q4, Q8, Q8Sparse])
def test_inputs_that_are_stored_late(qa, producer, cache, graphed):
    length, n = 700, 3
    w = (1 + 0.1 * rows(1, D), 1 + 0.1 * rows(2, D))
    src = rows(5, n, HQ + 2 * HKV, D)  # of a step: q, k, v behind each other
    got = []
    for late in (False, True):
        c, side = cache(qa, length, length + 10), torch.cuda.Stream()
        try:
            at = torch.zeros(1, HQ + 2 * HKV, D, device="cuda", dtype=torch.bfloat16)
            toks = at[:, :HQ], at[:, HQ:HQ + HKV], at[:, HQ + HKV:]
            outs = torch.zeros(n, 1, HQ, D, device="cuda", dtype=torch.bfloat16)
            torch.cuda.synchronize()

            def calls(stream):
                for i in range(n):
                    if late:
                        assert producer(at.data_ptr(), src[i].data_ptr(), at.numel() // 8, 100_000, stream.cuda_stream) == 0
                    else:
                        with torch.cuda.stream(stream):
                            at.copy_(src[i:i + 1])
                    c.step(i % 2, length + i // 2, toks, w, outs[i], stream)

            qa.qa_set_early_reads(not late)
            try:
                if graphed:
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph, stream=side):
                        calls(side)
                    torch.cuda.synchronize()
                    graph.replay()
                else:
                    calls(side)
            finally:
                qa.qa_set_early_reads(True)
            torch.cuda.synchronize()
            assert c.error()[0] == 0
            got.append(outs)
        finally:
            c.close()
    assert torch.equal(*got) and got[0].abs().sum() > 0


def test_a_chain_of_steps_without_overlap(qa):
    """The same bits with and without, whatever is recorded of the steps before."""
    w = (1 + 0.1 * rows(1, D), 1 + 0.1 * rows(2, D))
    toks = [(rows(50 + 3 * i, 1, HQ, D), rows(51 + 3 * i, 1, HKV, D), rows(52 + 3 * i, 1, HKV, D)) for i in range(24)]
    for cache in (Bf16, Q4, Q8, Q8Sparse):
        got = []
        for pattern in ((True,), (False,), (True, True, False, False, False)):
            c = cache(qa, 2000, 2100)
            try:
                outs = torch.zeros(24, 1, HQ, D, device="cuda", dtype=torch.bfloat16)
                for i, t in enumerate(toks):
                    qa.qa_set_early_reads(pattern[i % len(pattern)])
                    c.step(i // 2 % 2, 2000 + i // 4 * 2 + i % 2, t, w, outs[i], torch.cuda.current_stream())
                torch.cuda.synchronize()
                assert c.error()[0] == 0
                got.append(outs)
            finally:
                qa.qa_set_early_reads(True)
                c.close()
        assert all(torch.equal(got[0], x) for x in got[1:]), cache


def test_refusals(qa):
    for bad in (-1, 2):
        assert qa.lib.qa_set_early_reads(bad) == 1
