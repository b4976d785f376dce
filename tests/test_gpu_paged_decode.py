"""The bf16 decoding kernel (at most 128 rows of no more tokens than requests) with groups
of nine to sixteen query heads, which take row tiles of sixteen, and with more requests
than a warp has lanes, against the float64 oracle (tolerances: test_gpu_paged)."""
import pytest

from .test_gpu_paged import Batch

pytestmark = pytest.mark.gpu

BUSY = [(1, 1), (2, 1030), (0, 7), (1, 300), (1, 129), (0, 0), (2, 64), (0, 900)]
IDLE = [(0, 5 * r) for r in range(33)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [9, 11, 16])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 100)])
@pytest.mark.parametrize("lens", [BUSY, IDLE + BUSY], ids=["8", "41"])
def test_decode_wide_groups_masks(d, G, causal, window, lens):
    b = Batch(lens, 2 * G, 2, d, 48, "bf16", seed=G + window, L=2, layer=1, layout="fused")
    assert b.N <= len(lens) and b.N * G <= 128
    b.run(causal, window)
    b.check(causal, window)


@pytest.mark.parametrize("G", [4, 12])
@pytest.mark.parametrize("B", [1, 7, 16, 100, 128, 1000])
def test_decode_many_requests_page_sizes(G, B):
    b = Batch(IDLE + BUSY + IDLE * 8, 2 * G, 2, 128, B, "bf16", seed=B)
    assert b.N * G <= 128 and len(b.lens) > 256
    b.run()
    b.check()
