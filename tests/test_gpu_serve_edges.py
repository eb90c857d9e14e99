"""The operators around the attention in calls that an earlier form of them answered wrongly."""
import numpy as np
import pytest

from tests.test_gpu_serve import bf16, f32, fill, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pisa():
    import block_sparse_long_pisa_b200 as m
    return m


# ----------------------------------------------------------------------------- streams

BUSY = 20_000_000   # cycles that a stream is held for: about 10 ms, a thousand launches


def test_cache_read_on_a_stream_while_the_current_one_is_busy(pisa):
    """The outputs that the call makes are zeroed before its rows come, whatever the current stream still has to do."""
    import torch
    rng = np.random.default_rng(71)
    cache, _, _ = fill(pisa, rng, pisa.CacheShape(3, 2, 256, 128))
    ws, start, count = pisa.new_cache_workspace("cuda"), i32([0, 9, 200]), i32([50, 0, 33])
    want = pisa.cache_read(cache, 50, ws, start=start, count=count)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    got = pisa.cache_read(cache, 50, ws, start=start, count=count, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool(want[0].any())
