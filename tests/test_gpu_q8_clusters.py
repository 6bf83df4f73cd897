"""Steps of the 8-bit cache whose sequences are shared by several thread blocks, where a
position is outside the cache: those thread blocks leave together, the others go on."""
import pytest
import torch

from gpu_util import f64
from test_gpu_q8 import Cache, close, qa  # noqa: F401

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("hq,hkv,d,cap", [(8, 2, 128, 2100), (8, 2, 64, 6000), (3, 3, 128, 9000)])
@pytest.mark.parametrize("blocks", [0, 2])
def test_positions_outside_the_cache_among_clusters(qa, hq, hkv, d, cap, blocks):
    lens = [cap - 2, 700, 64, 1000]
    with Cache(qa, 4, hq, hkv, d, cap) as c:
        c.fill(lens, 3)
        for bad in ([1], [0, 2], [3], [0, 1, 2, 3]):
            at = [(-1, cap, 1 << 30, -(1 << 31))[b] if b in bad else p for b, p in enumerate(lens)]
            q, k, v = c.tokens(4, 8)
            out = torch.full_like(q, 5.0)
            lists = torch.full((4, hkv, 2), 77, dtype=torch.int32, device="cuda")
            if blocks:
                qa.qa_q8_sparse_step_device_positions(c.h, 0, 4, ints(at), 2, q, k, v, None, None, out, lists)
            else:
                qa.qa_q8_decode_step_device_positions(c.h, 0, 4, ints(at), q, k, v, None, None, out)
            assert qa.qa_q8_get_device_error(c.h)[0] == 8
            good = [b for b in range(4) if b not in bad]
            assert all((out[b] == 5.0).all() and (not blocks or (lists[b] == -1).all()) for b in bad)
            c.ref.write(lens, [int(b in good) for b in range(4)], f64(k)[good], f64(v)[good])
            for b in good:
                close(out[b:b + 1], *c.want(b, lens[b], q[b:b + 1].double(), lists[b].cpu().numpy() if blocks else None),
                      what=f"{bad}: sequence {b}")
        assert qa.qa_q8_get_device_error(c.h) == (0, 0)
