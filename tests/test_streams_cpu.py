"""Where a call that is given a stream makes its own tensors: on that stream. No GPU: the streams here are stand-ins, the
tensors live on the CPU, and a call ends where its checks find that out."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")
pisa = pytest.importorskip("block_sparse_long_pisa_b200")
from torch.utils._python_dispatch import TorchDispatchMode

MAKES = ("empty", "zeros", "new_empty", "empty_like", "zero_", "fill_", "empty_strided", "zeros_like", "new_zeros")


class Stream:
    device = "cpu"
    cuda_stream = 0


class Made(TorchDispatchMode):
    """The streams that tensors were made or filled on, in order."""

    def __init__(self, where):
        super().__init__()
        self.where, self.seen = where, []

    def __torch_dispatch__(self, func, types_, args=(), kwargs=None):
        if func.overloadpacket.__name__ in MAKES:
            self.seen.append(self.where[-1])
        return func(*args, **(kwargs or {}))


@pytest.fixture()
def made(monkeypatch):
    """run(call, stream) -> the streams of the tensors that the call makes."""
    where = [None]

    @contextlib.contextmanager
    def on(stream):
        where.append(stream)
        yield
        where.pop()

    class Torch(types.ModuleType):
        def __getattr__(self, name):
            return getattr(torch, name)

    fake = Torch("torch")
    fake.cuda = types.SimpleNamespace(stream=on, current_stream=lambda device=None: where[-1] or side)
    side = Stream()
    monkeypatch.setattr(pisa, "_torch_module", fake)

    def run(call):
        with Made(where) as m, pytest.raises(ValueError, match="CUDA tensor"):
            call(side)
        assert m.seen
        return [s is side for s in m.seen]

    return run


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_cache_read_fills_its_outputs_on_its_stream(made):
    cache = pisa.new_cache(pisa.CacheShape(2, 1, 64, 64), "cpu")
    n, ws = torch.zeros(2, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    for kw in (dict(count=n), dict(start=n), dict()):
        assert all(made(lambda s: pisa.cache_read(cache, 5, ws, stream=s, **kw)))


def test_calls_make_their_outputs_and_scratch_on_their_stream(made):
    nr = pisa.NormRopeShape(1, 2, 2, 1, 64, 0)
    xq, xk, w = bf16(1, 2, 2, 64), bf16(1, 2, 1, 64), torch.ones(64)
    assert all(made(lambda s: pisa.qk_norm_rope(nr, xq, xk, None, None, stream=s)))
    grads = (bf16(1, 2, 2, 64), bf16(1, 1, 2, 64))
    seen = made(lambda s: pisa.qk_norm_rope_backward(nr, xq, xk, None, None, *grads, w, w, stream=s))
    assert len(seen) == 5 and all(seen)              # dXq, dXk, dwq, dwk and the partial sums
    s = pisa.TreeShape(1, 2, 1, 2, 64, 64)
    q, kv, mask, n = bf16(1, 2, 2, 64), bf16(1, 1, 2, 64), torch.zeros((1, 2), dtype=torch.int64), torch.zeros(1, dtype=torch.int32)
    cache, ws = pisa.new_cache(pisa.CacheShape(1, 1, 64, 64), "cpu"), torch.zeros(4096, dtype=torch.uint8)
    seen = made(lambda st: pisa.tree_attention(s, cache, q, kv, kv, mask, n, ws, stream=st))
    assert len(seen) == 2 and all(seen)
