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


def test_scratch_of_the_gradients_is_kept_from_others(pisa):
    """Gradient calls on another stream make their own workspace: what the current stream allocates and writes after them
    does not meet it."""
    import torch
    rng = np.random.default_rng(72)
    B, N, Hq, Hkv, D = 1, 1024, 4, 2, 64
    x = bf16(rng, B, N, Hq + 2 * Hkv, D)
    nr, w = pisa.NormRopeShape(B, N, Hq, Hkv, D, D), f32(1 + 0.1 * rng.standard_normal(D))
    rope = (nr, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], i32(np.arange(N)[None]), f32(100.0 ** (-np.arange(32) / 32)))
    Q, K = pisa.qk_norm_rope(*rope, w, w)
    V = x[:, :, Hq + Hkv:].transpose(1, 2).contiguous()
    shape = pisa.Shape(B, Hq, Hkv, N, N, D, 64, 4, 4, causal=1)
    O, lse, idx = pisa.forward(shape, Q, K, V, pisa.new_workspace(shape, "cuda"), idx=True)
    dO = bf16(rng, B, Hq, N, D)

    def grads(stream=None):
        return [*pisa.sparse_attention_backward(shape, Q, K, V, O, lse, dO, idx, stream=stream),
                *pisa.qk_norm_rope_backward(*rope, dO, K, w, w, stream=stream)]

    want = grads()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    got = grads(side)
    sizes = (pisa.backward_workspace_size(shape), pisa.norm_rope_workspace_size(nr))
    junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(junk) == 8


def test_outputs_made_on_another_stream(pisa):
    """Outputs of a call on another stream do not take memory that the current stream has yet to read."""
    import torch
    from tests.test_gpu_serve import tmask, tree_inputs
    case = (2, 4, 2, 5, 512, 128, 1, 64, 0, 0, 0, [500, 77], "tree")
    s, cache, k, v, q, dk, dv, mask, lens, idx = tree_inputs(pisa, case, 73)
    ws, m, n, side = pisa.new_tree_workspace(s, "cuda"), tmask(mask), i32(lens), torch.cuda.Stream()
    want, want_lse = pisa.tree_attention(s, cache, q, dk, dv, m, n, ws)
    mine, kept = torch.full_like(q, 5.0), torch.empty_like(q)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    kept.copy_(mine)
    del mine                                          # to the current stream's pool, still to be read there
    O, lse = pisa.tree_attention(s, cache, q, dk, dv, m, n, ws, stream=side)
    torch.cuda.synchronize()
    assert bool((kept == 5.0).all()) and torch.equal(O, want) and torch.equal(lse, want_lse)
