"""The handle of a K/V cache gives a call its buffers as they are at the call. No GPU: only addresses are looked at."""
import pytest

torch = pytest.importorskip("torch")
pisa = pytest.importorskip("block_sparse_long_pisa_b200")


def caches():
    for fmt in (pisa.CACHE_E4M3, pisa.CACHE_BF16):
        yield pisa.new_cache(pisa.CacheShape(2, 3, 64, 64, fmt), "cpu")


def test_buffers_cannot_be_replaced():
    for cache in caches():
        for name in ("k", "v", "k_exp", "v_exp", "shape", "device"):
            with pytest.raises(AttributeError):
                setattr(cache, name, getattr(cache, name))


def pointers(cache, monkeypatch):
    """What a call of cache_read hands to the library."""
    seen = []

    def launch(where, call, stream, named, args):
        seen.append(args)

    monkeypatch.setattr(pisa, "_launch", launch)
    pisa.cache_read(cache, 1, torch.zeros(256, dtype=torch.uint8))
    return tuple(seen[0][2:6])


def test_addresses_are_those_of_the_call(monkeypatch):
    for cache in caches():
        have = [t for t in (cache.k, cache.v, cache.k_exp, cache.v_exp) if t is not None]
        for t in have:
            before = t.data_ptr()
            other = torch.empty_like(t)
            t.set_(other)                           # a buffer moves: the old memory may be gone
            assert t.data_ptr() == other.data_ptr() != before
            want = tuple(None if x is None else x.data_ptr() for x in (cache.k, cache.v, cache.k_exp, cache.v_exp))
            assert pointers(cache, monkeypatch) == want


def test_buffers_of_another_shape_are_refused(monkeypatch):
    for i in range(4):
        for cache in caches():
            t = (cache.k, cache.v, cache.k_exp, cache.v_exp)[i]
            if t is None:
                continue
            t.set_(torch.empty((2, 3, 32, *t.shape[3:]), dtype=t.dtype))
            with pytest.raises(ValueError, match=("k", "v", "k_exp", "v_exp")[i]):
                pointers(cache, monkeypatch)
