"""The operators around the attention against their 64-bit oracle, at the sizes and masks where they
can go wrong, and together as a serving and a training step use them.

Tolerances. A bf16 result is off by at most half a step, 2^-8 relative. fp32 arithmetic adds:
  * norm and rotation: about 12 roundings of 2^-24 of the two products that a value is made of and of
    the row's scale: 2^-19 of the row's largest value;
  * gradients: the same of r (|dn| + |x r| mean|dn x r|); the weights' sums 2^-19 of
    the sum of (|dy_a| + |dy_b|) |x r| (a term's two rotated products may cancel; their errors, and those
    of cos and sin, 2^-24 of each, do not);
  * node means: at most 2^-24 per addition, 2^-19 of the mean |x| for the sizes here;
  * attention: each probability is rounded to bf16 once (2^-8; fp16 rounds less) and its score is off
    by the products' fp32 accumulation, 2^-18 of sum |q k| scale, natural units:
    |dO| <= 2^-8 |O| + (2^-8 + 2 e) sum p|v|, |dLSE| <= e + 2^-20 |LSE| + 2^-18, e = 2^-18 sum |q k| scale.
Bytes, exponents and rows read back are exact.
"""
import dataclasses
import math

import numpy as np
import pytest

import oracle
from oracle import serve_oracle as so

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pisa():
    import block_sparse_long_pisa_b200 as m
    return m


def bf16(rng, *shape, scale=1.0):
    import torch
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(torch.bfloat16).cuda()


def host(t):
    return t.detach().to("cpu").double().numpy()


def f32(x):
    import torch
    return torch.from_numpy(np.asarray(x, np.float32)).cuda()


def i32(x):
    import torch
    return torch.from_numpy(np.asarray(x, np.int32)).cuda()


# ----------------------------------------------------------------------------- norm and rotation

NR_CASES = [
    # B, T, Hq, Hkv, D, R, interleaved, weights, far, packed
    (1, 1, 1, 1, 64, 64, 0, 1, 0, 1),
    (1, 1, 1, 1, 128, 128, 1, 1, 7, 0),
    (64, 1, 32, 8, 128, 128, 0, 1, 131072, 1),
    (3, 7, 5, 1, 128, 112, 0, 1, 1000000, 1),
    (2, 33, 12, 4, 64, 48, 0, 1, 0, 1),
    (2, 33, 12, 4, 64, 16, 1, 0, 5, 1),
    (1, 700, 8, 8, 128, 32, 1, 1, 2 ** 31 - 800, 0),
    (1, 50, 3, 2, 128, 0, 0, 1, 0, 1),
    (2, 1000, 40, 8, 64, 64, 0, 1, 3, 1),
    (1, 12000, 4, 2, 128, 128, 0, 1, 0, 1),
    (1, 600, 33, 2, 128, 128, 0, 0, -20000, 1),
]


def nr_inputs(case, seed):
    import torch
    B, T, Hq, Hkv, D, R, inter, weights, far, packed = case
    rng = np.random.default_rng(seed)
    if packed:
        x = bf16(rng, B, T, Hq + 2 * Hkv, D)
        xq, xk = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]
    else:
        xq, xk = bf16(rng, B, T, Hq, D), bf16(rng, B, Hkv, T, D).transpose(1, 2)
    xq.mul_(torch.exp2(torch.arange(Hq, device="cuda") % 5 - 2).to(torch.bfloat16)[:, None])   # heads of unlike size
    wq, wk = (1 + 0.3 * rng.standard_normal(D), 1 + 0.3 * rng.standard_normal(D)) if weights else (None, None)
    pos = (np.int64(far) + np.arange(T)[None] + 3 * np.arange(B)[:, None]).astype(np.int32)
    fr = np.float32(10000.0) ** (-2.0 * np.arange(R // 2) / max(1, R))
    return rng, xq, xk, wq, wk, pos, fr.astype(np.float32)


@pytest.mark.parametrize("case", NR_CASES)
def test_norm_rope(pisa, case):
    B, T, Hq, Hkv, D, R, inter, weights, far, packed = case
    _, xq, xk, wq, wk, pos, fr = nr_inputs(case, 11)
    s = pisa.NormRopeShape(B, T, Hq, Hkv, D, R, inter, 1e-6)
    Q, K = pisa.qk_norm_rope(s, xq, xk, i32(pos), f32(fr), None if wq is None else f32(wq), None if wk is None else f32(wk))
    for got, x, w in ((Q, xq, wq), (K, xk, wk)):
        w = None if w is None else np.float32(w)
        ref = so.norm_rope(host(x), w, pos, fr, R, inter, np.float32(1e-6))
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * np.abs(ref).max(-1, keepdims=True) * 2
        err = np.abs(host(got) - ref)
        assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("case", NR_CASES)
def test_norm_rope_backward(pisa, case):
    import torch
    B, T, Hq, Hkv, D, R, inter, weights, far, packed = case
    rng, xq, xk, wq, wk, pos, fr = nr_inputs(case, 12)
    dq, dk = bf16(rng, B, Hq, T, D), bf16(rng, B, Hkv, T, D)
    s = pisa.NormRopeShape(B, T, Hq, Hkv, D, R, inter, 1e-6)
    tq, tk = (None, None) if wq is None else (f32(wq), f32(wk))
    grad = torch.full((B, T, Hq + 2 * Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    out = pisa.qk_norm_rope_backward(s, xq, xk, i32(pos), f32(fr), dq, dk, tq, tk, dXq=grad[:, :, :Hq],
                                     dXk=grad[:, :, Hq:Hq + Hkv])
    assert bool((grad[:, :, Hq + Hkv:] == 7.0).all())                   # the values' part is not touched
    for dx, dw, x, w, dy in ((out[0], out[2], xq, wq, dq), (out[1], out[3], xk, wk, dk)):
        w = None if w is None else np.float32(w)
        rx, rw, size = so.norm_rope_backward(host(x), w, pos, fr, R, inter, np.float32(1e-6), host(dy))
        r = 1 / np.sqrt((host(x) ** 2).mean(-1, keepdims=True) + 1e-6)
        big = r * np.abs(host(dy)).max() * (1.0 if w is None else np.abs(w).max()) * 2 * (1 + np.abs(host(x) * r).max(-1, keepdims=True))
        err = np.abs(host(dx) - rx)
        assert (err <= 2.0 ** -8 * np.abs(rx) + 2.0 ** -19 * big).all()
        if w is None:
            assert dw is None
        else:
            assert (np.abs(host(dw) - rw) <= 2.0 ** -19 * size).all()
    again = pisa.qk_norm_rope_backward(s, xq, xk, i32(pos), f32(fr), dq, dk, tq, tk)
    assert torch.equal(again[0], out[0]) and torch.equal(again[1], out[1])
    if tq is not None:
        assert torch.equal(again[2], out[2]) and torch.equal(again[3], out[3])


def test_norm_rope_without_eps(pisa):
    """eps = 0: rows that do not exist (the last tile's) add nothing to the weights' gradient."""
    rng = np.random.default_rng(4)
    B, T, Hq, Hkv, D = 1, 37, 3, 1, 64
    xq, xk, dq, dk = bf16(rng, B, T, Hq, D), bf16(rng, B, T, Hkv, D), bf16(rng, B, Hq, T, D), bf16(rng, B, Hkv, T, D)
    s = pisa.NormRopeShape(B, T, Hq, Hkv, D, D, 0, 0.0)
    pos, fr = np.arange(T)[None].astype(np.int32), np.float32(1.0) / (1 + np.arange(32, dtype=np.float32))
    w = f32(np.ones(D))
    _, _, dwq, dwk = pisa.qk_norm_rope_backward(s, xq, xk, i32(pos), f32(fr), dq, dk, w, w)
    for dw, x, dy in ((dwq, xq, dq), (dwk, xk, dk)):
        _, rw, size = so.norm_rope_backward(host(x), None, pos, fr, D, 0, 0.0, host(dy))
        assert (np.abs(host(dw) - rw) <= 2.0 ** -19 * size).all()


def test_norm_rope_rows_that_are_not_finite_stay_alone(pisa):
    """A NaN or an infinity in one row leaves every other row as it was; a zero row gives zeros."""
    import torch
    rng = np.random.default_rng(5)
    B, T, Hq, Hkv, D = 1, 9, 4, 2, 128
    xq, xk = bf16(rng, B, T, Hq, D), bf16(rng, B, T, Hkv, D)
    s = pisa.NormRopeShape(B, T, Hq, Hkv, D, 64)
    pos, fr = i32(np.arange(T)[None]), f32(1.0 / (1 + np.arange(32)))
    Q0, K0 = pisa.qk_norm_rope(s, xq, xk, pos, fr)
    xq[0, 3, 1, 70] = float("nan")
    xq[0, 5, 2, 3] = float("inf")
    xk[0, 2, 1] = 0
    Q, K = pisa.qk_norm_rope(s, xq, xk, pos, fr)
    assert bool(torch.isnan(Q[0, 1, 3]).all()) and bool(torch.isnan(Q[0, 2, 5]).any()) and bool((K[0, 1, 2] == 0).all())
    Q[0, 1, 3], Q[0, 2, 5], K[0, 1, 2] = Q0[0, 1, 3], Q0[0, 2, 5], K0[0, 1, 2]
    assert torch.equal(Q, Q0) and torch.equal(K, K0)


def test_norm_rope_refusals(pisa):
    import torch
    rng = np.random.default_rng(6)
    s = pisa.NormRopeShape(1, 4, 2, 1, 64, 64)
    xq, xk, pos, fr = bf16(rng, 1, 4, 2, 64), bf16(rng, 1, 4, 1, 64), i32(np.arange(4)[None]), f32(np.ones(32))
    for bad in (dict(Xq=xq.float()), dict(Xq=xq[:, :3]), dict(Xq=xq.transpose(2, 3).contiguous().transpose(2, 3)),
                dict(Xk=xk.cpu()), dict(pos=pos.long()), dict(pos=pos.cpu()), dict(inv_freq=fr[:31]),
                dict(wq=f32(np.ones(63))), dict(Q=xq)):
        a = dict(Xq=xq, Xk=xk, pos=pos, inv_freq=fr)
        a.update(bad)
        with pytest.raises((ValueError, pisa.PisaError)):
            pisa.qk_norm_rope(s, **a)
    wide = bf16(rng, 1, 4, 2, 68)[..., :64]                              # strides not multiples of 8
    with pytest.raises(pisa.PisaError):
        pisa.qk_norm_rope(s, wide, xk, pos, fr)
    dq, dk = bf16(rng, 1, 2, 4, 64), bf16(rng, 1, 1, 4, 64)
    with pytest.raises(pisa.PisaError):                                  # gradients that overlap in themselves
        pisa.qk_norm_rope_backward(s, xq, xk, pos, fr, dq, dk, dXq=torch.empty_like(xq[:, :, :1]).expand(-1, -1, 2, -1))


def test_norm_rope_broadcast_input(pisa):
    """One head's input repeated by a stride of 0: the outputs are those of a copy."""
    import torch
    rng = np.random.default_rng(7)
    one = bf16(rng, 2, 5, 1, 64)
    s = pisa.NormRopeShape(2, 5, 3, 3, 64, 64)
    pos, fr = i32(np.arange(10).reshape(2, 5)), f32(1.0 / (1 + np.arange(32)))
    wide = one.expand(-1, -1, 3, -1)
    a = pisa.qk_norm_rope(s, wide, wide, pos, fr)
    b = pisa.qk_norm_rope(s, wide.contiguous(), wide.contiguous(), pos, fr)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ----------------------------------------------------------------------------- the cache

def raw(cache):
    """Bytes of the cache's buffers, on the host."""
    import torch
    out = [cache.k.view(torch.uint8).cpu().numpy().copy(), cache.v.view(torch.uint8).cpu().numpy().copy()]
    return out + ([cache.k_exp.cpu().numpy().copy(), cache.v_exp.cpu().numpy().copy()] if cache.k_exp is not None else [])


def special_rows(rng, D):
    """Rows that test the quantiser's borders, bf16-exact."""
    import torch
    g = so.e4m3_grid()
    rows = [np.zeros(D), np.full(D, -0.0)]
    for k in (-126, -60, -8, 0, 1, 30, 119):
        x = rng.choice(g, D) * rng.choice([-1, 1], D)
        x[0] = 448
        rows += [x * 2.0 ** k]
        y = rng.choice((g[1:] + g[:-1]) / 2, D)                          # ties
        y[1] = 448 if k % 2 else 449 + 7
        rows += [y * 2.0 ** k]
    big = rng.standard_normal(D)
    big[3] = 3.3895e38                                                   # bf16's largest
    tiny = np.zeros(D)
    tiny[2] = 2.0 ** -133                                                # bf16's smallest subnormal
    rows += [big, tiny, np.full(D, 1.75), np.full(D, 1.7578125)]
    t = torch.from_numpy(np.stack(rows).astype(np.float32)).to(torch.bfloat16)
    return t


@pytest.mark.parametrize("D", [64, 128])
def test_cache_write_borders(pisa, D):
    import torch
    rng = np.random.default_rng(D)
    rows = special_rows(rng, D)
    n = rows.shape[0]
    K = rows[None, None].cuda()
    V = rows.flip(0)[None, None].cuda().contiguous()
    V[0, 0, 3, 5], V[0, 0, 4, 6], V[0, 0, 5, D - 1] = float("nan"), float("inf"), float("-inf")
    cache = pisa.new_cache(pisa.CacheShape(1, 1, n + 5, D), "cuda")
    ws = pisa.new_cache_workspace("cuda")
    pisa.cache_write(cache, K, V, ws, start=i32([2]))
    assert pisa.check_status(ws) == (pisa.OK, 0)
    k, v, ke, ve = raw(cache)
    for got, ge, x in ((k, ke, K), (v, ve, V)):
        q, e = so.quantise_rows(host(x)[0, 0])
        assert np.array_equal(ge[0, 0, 2:2 + n], e)
        same = got[0, 0, 2:2 + n] == q
        assert (same | ((got[0, 0, 2:2 + n] | q) == 0x80)).all()         # the sign of a zero aside
    back, vback = pisa.cache_read(cache, n, ws, start=i32([2]))
    # exact where bf16 has the value: a byte of 2^-9 at e = 1 is 2^-135, below bf16's 2^-133, and is rounded
    val = torch.from_numpy(so.row_values(k[0, 0, 2:2 + n], ke[0, 0, 2:2 + n])).float().to(torch.bfloat16)
    assert np.array_equal(host(back)[0, 0], host(val), equal_nan=True)
    assert torch.isnan(vback[0, 0, 3:6]).all() and not torch.isnan(vback[0, 0, 6:]).any()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("B, H, T, cap, D", [(1, 1, 1, 1, 64), (1, 1, 1, 64, 128), (5, 3, 17, 40, 128), (3, 2, 301, 512, 64),
                                             (64, 8, 1, 96, 128), (2, 1, 1000, 1000, 128)])
def test_cache_ragged_write_and_read(pisa, fmt, B, H, T, cap, D):
    import torch
    rng = np.random.default_rng(T + D + fmt)
    cache = pisa.new_cache(pisa.CacheShape(B, H, cap, D, fmt), "cuda")
    ws = pisa.new_cache_workspace("cuda")
    pisa.cache_write(cache, bf16(rng, B, H, cap, D), bf16(rng, B, H, cap, D), ws)          # full to begin with
    before = raw(cache)
    packed = bf16(rng, B, T, 2 * H, D)
    K, V = packed[:, :, :H].transpose(1, 2), packed[:, :, H:].transpose(1, 2)
    start = rng.integers(0, cap - T + 1, B)
    count = rng.integers(0, T + 1, B)
    count[0] = T
    if B > 2:
        count[1] = 0
        start[2], count[2] = cap - T, T
    pisa.cache_write(cache, K, V, ws, start=i32(start), count=i32(count))
    assert pisa.check_status(ws) == (pisa.OK, 0)
    after = raw(cache)
    kh, vh = host(K), host(V)
    want = [x.copy() for x in before]
    for b in range(B):
        a, n = start[b], count[b]
        for side, x in ((0, kh), (1, vh)) if n else ():
            if fmt == 1:
                q, e = so.quantise_rows(x[b, :, :n])
                want[side][b, :, a:a + n], want[2 + side][b, :, a:a + n] = q, e
            else:
                t = torch.from_numpy(x[b, :, :n].copy()).to(torch.bfloat16)
                want[side][b, :, a:a + n] = t.view(torch.uint8).numpy()
    for x, y in zip(after, want):
        assert np.array_equal(np.where(x == 0x80, 0, x), np.where(y == 0x80, 0, y))
    marker = torch.full((B, H, T, D), 3.0, dtype=torch.bfloat16, device="cuda")
    rk, rv = pisa.cache_read(cache, T, ws, start=i32(start), count=i32(count), K=marker, V=marker.clone())
    for b in range(B):
        a, n = start[b], count[b]
        for got, side in ((rk, 0), (rv, 1)):
            assert bool((got[b, :, n:] == 3.0).all())
            if n == 0:
                continue
            x = after[side][b, :, a:a + n]
            ref = so.row_values(x, after[2 + side][b, :, a:a + n]) if fmt == 1 else \
                host(torch.from_numpy(x.copy()).view(torch.bfloat16))
            assert np.array_equal(host(got)[b, :, :n], ref)


def test_cache_ranges_that_do_not_fit_are_left_and_recorded(pisa):
    rng = np.random.default_rng(1)
    B, H, T, cap, D = 6, 2, 4, 10, 64
    cache = pisa.new_cache(pisa.CacheShape(B, H, cap, D), "cuda")
    ws = pisa.new_cache_workspace("cuda")
    before = raw(cache)
    for start, count in (([0, -1, 7, 2147483647, 0, 6], [4, 1, 4, 4, 5, 4]), ([0, 0, 0, 10, 11, 6], [4, -1, 0, 0, 0, 4])):
        K, V = bf16(rng, B, H, T, D), bf16(rng, B, H, T, D)
        pisa.cache_write(cache, K, V, ws, start=i32(start), count=i32(count))
        st, detail = pisa.check_status(ws)
        assert st == pisa.ERR_BAD_INDEX and detail >> 8 == 6
        after = raw(cache)
        for b in (1, 2, 3, 4):
            assert all(np.array_equal(x[b], y[b]) for x, y in zip(before, after)), b
        q, e = so.quantise_rows(host(K)[5])
        assert np.array_equal(after[2][5, :, 6:10], e)
        out = bf16(rng, B, H, T, D)
        keep = host(out).copy()
        pisa.cache_read(cache, T, ws, start=i32(start), count=i32(count), K=out, V=out.clone())
        assert pisa.check_status(ws)[0] == pisa.ERR_BAD_INDEX
        assert np.array_equal(host(out)[1:5], keep[1:5])
    assert pisa.check_status(ws) == (pisa.OK, 0)


def test_cache_refusals(pisa):
    import torch
    rng = np.random.default_rng(2)
    cache = pisa.new_cache(pisa.CacheShape(2, 2, 64, 64), "cuda")
    ws = pisa.new_cache_workspace("cuda")
    K = bf16(rng, 2, 2, 3, 64)
    for a in (dict(K=K[:1]), dict(K=K.float()), dict(V=K[:, :, :2]), dict(K=K.cpu()), dict(start=i32([0])),
              dict(count=torch.zeros(2, dtype=torch.int64, device="cuda")), dict(ws=ws[:100]), dict(ws=ws.float())):
        with pytest.raises((ValueError, pisa.PisaError)):
            pisa.cache_write(cache, **{**dict(K=K, V=K, ws=ws), **a})
    for tokens in (0, 65):
        with pytest.raises((ValueError, pisa.PisaError)):
            pisa.cache_read(cache, tokens, ws)
    s = cache.shape
    with pytest.raises(ValueError):
        pisa.Cache(s, cache.k, cache.v, None, None)
    with pytest.raises(ValueError):
        pisa.Cache(dataclasses.replace(s, format=pisa.CACHE_BF16), cache.k, cache.v)
    with pytest.raises(ValueError):
        pisa.cache_write(pisa.Cache(s, cache.k, None, cache.k_exp), K, K, ws)


def fill(pisa, rng, shape, scale=1.0, spread=0):
    """A cache full of random rows (rows of unlike size with `spread`), and its values in fp64."""
    import torch
    B, H, cap, D = shape.batch, shape.heads_kv, shape.capacity, shape.head_dim
    cache = pisa.new_cache(shape, "cuda")
    K, V = bf16(rng, B, H, cap, D, scale=scale), bf16(rng, B, H, cap, D, scale=scale)
    if spread:
        f = torch.from_numpy(2.0 ** rng.integers(-spread, spread + 1, (B, H, cap, 1))).to(torch.bfloat16).cuda()
        V = V * f
    pisa.cache_write(cache, K, V, pisa.new_cache_workspace("cuda"))
    if shape.format == pisa.CACHE_BF16:
        return cache, host(cache.k), host(cache.v)
    k, v, ke, ve = raw(cache)
    return cache, so.row_values(k, ke), so.row_values(v, ve)


@pytest.mark.parametrize("B, H, n, spare, D, blk, f", [(1, 1, 1, 0, 64, 64, 4), (2, 3, 37, 5, 128, 64, 4), (1, 2, 9, 0, 128, 128, 2),
                                                       (3, 1, 130, 70, 64, 64, 3), (1, 1, 6, 100, 128, 64, 80)])
def test_cache_pyramid(pisa, B, H, n, spare, D, blk, f):
    """Nodes against their means; an append from any length equals one call from zero bit for bit; rows
    past the length (garbage here) are not read."""
    import torch
    rng = np.random.default_rng(n)
    cap = (n + spare) * blk
    cache, kv, _ = fill(pisa, rng, pisa.CacheShape(B, H, cap, D))
    if spare:
        cache.k.view(torch.uint8)[:, :, n * blk:] = 0x7F
        cache.k_exp[:, :, n * blk:] = 255
    s = pisa.Shape(B, H, H, 1, n * blk, D, blk, f, 1, kv_capacity=cap)
    sizes, offs = pisa.level_layout(s)
    assert s.n_nodes == sum(sizes)
    pyr = torch.zeros((B, H, sum(sizes), D), device="cuda")
    pisa.cache_append_pyramid(s, cache, pyr, 0)
    got = host(pyr)
    for l, (size, off) in enumerate(zip(sizes, offs)):
        for c in range(size):
            lo, hi = min(c * f ** l, n) * blk, min((c + 1) * f ** l, n) * blk
            if hi == lo:
                assert not got[:, :, off + c].any()
                continue
            x = kv[:, :, lo:hi]
            assert (np.abs(got[:, :, off + c] - x.mean(2)) <= 2.0 ** -19 * np.abs(x).mean(2)).all(), (l, c)
    for cuts in ([n // 2], [n - 1], list(range(1, n, 7))):
        p2, old = torch.zeros_like(pyr), 0
        for c in sorted({c for c in cuts if 0 < c < n} | {n}):
            pisa.cache_append_pyramid(dataclasses.replace(s, seq_kv=c * blk), cache, p2, old)
            old = c * blk
        assert torch.equal(p2, pyr)
    pisa.cache_append_pyramid(s, cache, pyr, n * blk)                    # nothing new
    assert np.array_equal(host(pyr), got)


# ----------------------------------------------------------------------------- drafted tokens

def tree_bits(rng, B, T, kind):
    m = np.zeros((B, T), np.uint64)
    for b in range(B):
        rows = []
        for t in range(T):
            if kind == "chain":
                w = (1 << (t + 1)) - 1
            elif kind == "tree":
                w = (1 << t) | (rows[rng.integers(0, t)] if t else 0)
            elif kind == "none":
                w = 0
            else:
                w = int(rng.integers(0, 1 << 62)) | (int(rng.integers(0, 4)) << 62)   # bits past T too
            rows.append(w)
            m[b, t] = w
    return m


TREE_CASES = [
    # B, Hq, Hkv, T, cap, D, fmt, blk, seq, topk, perq, lens, mask
    (1, 1, 1, 1, 64, 64, 0, 64, 0, 0, 0, [0], "chain"),
    (1, 1, 1, 1, 64, 128, 1, 64, 0, 0, 0, [0], "none"),
    (1, 1, 1, 1, 64, 128, 1, 64, 0, 0, 0, [1], "none"),
    (2, 2, 1, 1, 128, 128, 1, 64, 0, 0, 0, [128, 63], "chain"),
    (2, 8, 2, 1, 1024, 128, 1, 64, 896, 5, 0, [1000, 896], "chain"),
    (2, 8, 2, 1, 1024, 128, 0, 64, 896, 5, 0, [1000, 897], "chain"),
    (3, 6, 2, 5, 704, 64, 1, 64, 640, 3, 0, [700, 300, 0], "tree"),
    (3, 6, 2, 5, 704, 64, 0, 64, 640, 3, 1, [700, 300, 0], "tree"),
    (1, 4, 1, 7, 512, 128, 1, 128, 384, 2, 0, [511], "any"),
    (1, 4, 1, 7, 512, 128, 0, 128, 384, 2, 1, [200], "any"),
    (4, 4, 2, 16, 320, 128, 1, 64, 0, 0, 0, [320, 0, 65, 191], "tree"),
    (4, 4, 2, 16, 320, 128, 0, 64, 0, 0, 0, [320, 0, 65, 191], "tree"),
    (1, 8, 1, 3, 192, 64, 1, 64, 128, 2, 0, [150], "none"),
    (1, 3, 3, 33, 256, 128, 1, 64, 0, 0, 0, [250], "tree"),
    (1, 6, 2, 33, 256, 64, 0, 64, 0, 0, 0, [17], "any"),
    (2, 8, 2, 17, 256, 128, 1, 64, 192, 2, 0, [230, 100], "tree"),
    (1, 4, 1, 64, 192, 128, 0, 64, 0, 0, 0, [190], "any"),
    (1, 4, 1, 64, 192, 128, 1, 64, 0, 0, 0, [190], "any"),
    (1, 5, 1, 64, 192, 64, 1, 64, 128, 2, 0, [131], "tree"),
    (2, 8, 2, 24, 448, 128, 0, 64, 384, 3, 0, [448, 70], "tree"),
    (2, 8, 2, 24, 448, 128, 1, 64, 384, 3, 0, [448, 70], "tree"),
    (1, 9, 3, 11, 320, 64, 1, 64, 0, 0, 0, [319], "tree"),
    (1, 6, 1, 64, 256, 128, 1, 128, 128, 1, 0, [200], "any"),
    (1, 6, 1, 64, 256, 64, 0, 64, 0, 0, 0, [129], "tree"),
    (3, 8, 1, 20, 8192, 128, 1, 64, 0, 0, 0, [8000, 0, 64], "chain"),
    (3, 4, 1, 16, 8192, 128, 0, 64, 0, 0, 0, [1, 8191, 4000], "tree"),
    (2, 3, 1, 9, 256, 64, 0, 64, 192, 1, 1, [192, 255], "tree"),
    (1, 1, 1, 2, 40960, 128, 1, 64, 0, 0, 0, [40001], "chain"),
    (1, 2, 1, 2, 20480, 64, 0, 128, 0, 0, 0, [20479], "chain"),
    (33, 2, 2, 2, 128, 64, 1, 64, 0, 0, 0, None, "tree"),
    (70, 4, 1, 1, 256, 128, 1, 64, 192, 2, 0, None, "chain"),
    # two row tiles of 16, unlike ones too; as many drafted tokens as rows
    (3, 5, 1, 5, 448, 128, 1, 64, 320, 4, 0, [400, 0, 130], "tree"),
    (2, 2, 1, 16, 256, 64, 1, 64, 0, 0, 0, [250, 1], "tree"),
    (1, 1, 1, 17, 256, 128, 1, 64, 0, 0, 0, [200], "any"),
    # several pieces to a run
    (200, 4, 2, 20, 192, 64, 1, 64, 0, 0, 0, None, "tree"),
    (200, 4, 2, 20, 192, 128, 0, 64, 0, 0, 0, None, "tree"),
    (120, 4, 1, 40, 320, 128, 1, 64, 128, 2, 0, None, "tree"),
    (120, 4, 1, 40, 320, 64, 0, 64, 128, 2, 0, None, "tree"),
    (300, 4, 1, 8, 192, 128, 1, 64, 0, 0, 0, None, "tree"),
]


def tree_inputs(pisa, case, seed, spread=0, qscale=1.0):
    import torch
    B, Hq, Hkv, T, cap, D, fmt, blk, seq, topk, perq, lens, kind = case
    rng = np.random.default_rng(seed)
    cache, k, v = fill(pisa, rng, pisa.CacheShape(B, Hkv, cap, D, fmt), spread=spread)
    lens = rng.integers(0, cap + 1, B) if lens is None else np.array(lens)
    s = pisa.TreeShape(B, Hq, Hkv, T, cap, D, fmt, blk, seq, topk, perq)
    q, dk, dv = bf16(rng, B, Hq, T, D, scale=qscale), bf16(rng, B, Hkv, T, D), bf16(rng, B, Hkv, T, D)
    mask = tree_bits(rng, B, T, kind)
    idx = None
    if topk:
        idx = np.full((B, s.hsel, 1, topk), -1, np.int32)
        for b in range(B):
            for h in range(s.hsel):
                n = topk if (b + h) % 3 else max(0, topk - 2)           # some rows are short
                pick = np.sort(rng.choice(seq // blk, min(n, seq // blk), replace=False))
                idx[b, h, 0, :len(pick)] = pick
    # what lies past the length is garbage
    for b in range(B):
        if fmt == 1:
            for t in (cache.k, cache.v):
                t.view(torch.uint8)[b, :, lens[b]:] = 0x7F
            cache.k_exp[b, :, lens[b]:] = 255
            cache.v_exp[b, :, lens[b]:] = 255
        else:
            cache.k[b, :, lens[b]:] = float("nan")
            cache.v[b, :, lens[b]:] = float("inf")
    return s, cache, k, v, q, dk, dv, mask, lens, idx


def tmask(mask):
    import torch
    return torch.from_numpy(mask.view(np.int64)).cuda()


def check_tree(s, O, lse, k, v, q, dk, dv, mask, lens, idx, what=""):
    ref, L, A, S = so.tree_attention(host(q), host(dk), host(dv), mask, k, v, lens, idx, block=s.block, seq_kv=s.seq_kv,
                                     topk=s.topk, per_qhead=bool(s.select_per_qhead), scale=s.scale)
    e = 2.0 ** -18 * S
    err = np.abs(host(O) - ref)
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * e[..., None]) * A
    assert (err <= tol).all(), (what, np.nanmax(err - tol), np.argwhere(~(err <= tol))[:5])
    got = host(lse)
    empty = np.isneginf(L)
    assert np.array_equal(np.isneginf(got), empty), what
    assert (host(O)[empty] == 0).all()
    dl = np.abs(got[~empty] - L[~empty])
    assert (dl <= e[~empty] + 2.0 ** -20 * np.abs(L[~empty]) + 2.0 ** -18).all(), (what, dl.max())


@pytest.mark.parametrize("case", TREE_CASES)
def test_tree_attention(pisa, case):
    import torch
    s, cache, k, v, q, dk, dv, mask, lens, idx = tree_inputs(pisa, case, 21)
    ws = pisa.new_tree_workspace(s, "cuda")
    ws[256:] = 0xFF                                                       # partials need no clearing
    args = (s, cache, q, dk, dv, tmask(mask), i32(lens), ws)
    O, lse = pisa.tree_attention(*args, idx=None if idx is None else i32(idx))
    assert pisa.check_status(ws) == (pisa.OK, 0)
    check_tree(s, O, lse, k, v, q, dk, dv, mask, lens, idx)
    O2, none = pisa.tree_attention(*args, idx=None if idx is None else i32(idx), lse=None)
    assert none is None and torch.equal(O, O2)


@pytest.mark.parametrize("case", [TREE_CASES[i] for i in (4, 10, 13, 17, 18, 19, 24)])
@pytest.mark.parametrize("spread, qscale", [(12, 1.0), (0, 30.0), (6, 1e-3), (30, 1e-9)])
def test_tree_attention_of_unlike_rows(pisa, case, spread, qscale):
    """Value rows from 2^-12 (2^-30) to 2^12 (2^30) of one another (the unit of O moves), peaked and flat scores."""
    s, cache, k, v, q, dk, dv, mask, lens, idx = tree_inputs(pisa, case, 22, spread, qscale)
    ws = pisa.new_tree_workspace(s, "cuda")
    O, lse = pisa.tree_attention(s, cache, q, dk, dv, tmask(mask), i32(lens), ws, idx=None if idx is None else i32(idx))
    check_tree(s, O, lse, k, v, q, dk, dv, mask, lens, idx)


@pytest.mark.parametrize("T, Hq, D", [(1, 4, 128), (5, 4, 64), (5, 4, 128), (20, 4, 64), (24, 8, 128)])
def test_tree_attention_of_a_nan_byte(pisa, T, Hq, D):
    """A cached byte that is a NaN is one: in V for its dim of every token, in K for all dims; other sequences and
    heads keep their bits."""
    import torch
    case = (2, Hq, 2, T, 256, D, 1, 64, 0, 0, 0, [200, 170], "chain")
    s, cache, k, v, q, dk, dv, mask, lens, idx = tree_inputs(pisa, case, 23)
    ws = pisa.new_tree_workspace(s, "cuda")
    run = lambda: pisa.tree_attention(s, cache, q, dk, dv, tmask(mask), i32(lens), ws)[0]
    base = run()
    assert not torch.isnan(base).any()
    for t, dims in ((cache.v, [3]), (cache.k, list(range(D)))):
        byte = t.view(torch.uint8)[1, 0, 77, 3]
        kept = int(byte)
        byte.fill_(0xFF)
        O = run()
        bad = torch.zeros_like(O, dtype=torch.bool)
        bad[1, :Hq // 2, :, dims] = True
        assert torch.equal(torch.isnan(O), bad) and torch.equal(O[~bad], base[~bad])
        byte.fill_(kept)
    assert pisa.check_status(ws) == (pisa.OK, 0)



@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T, Hq", [(5, 1), (5, 2), (8, 4), (9, 4), (40, 2), (40, 4)])
def test_drafts_that_are_not_attended_do_not_touch_a_token(pisa, fmt, T, Hq):
    """Drafted token 2 holds NaN keys and values, token 3 infinite values: the tokens that attend
    neither are as if both held zeros; those that do see a NaN."""
    import torch
    case = (1, Hq, 1, T, 256, 128, fmt, 64, 0, 0, 0, [200], "chain")
    s, cache, k, v, q, dk, dv, mask, lens, idx = tree_inputs(pisa, case, 23)
    for t in range(T):
        mask[0, t] = np.uint64((1 << t) | (3 if t < 4 else 0b10011))
    mask[0, T - 1] = np.uint64(0b00110)
    ws = pisa.new_tree_workspace(s, "cuda")
    dk[0, 0, 2], dv[0, 0, 2], dv[0, 0, 3, 7] = 0, 0, 0
    dv[0, 0, 3] = 0
    clean, lc = pisa.tree_attention(s, cache, q, dk, dv, tmask(mask), i32(lens), ws)
    dk[0, 0, 2], dv[0, 0, 2] = float("nan"), float("nan")
    dv[0, 0, 3] = float("inf")
    O, l = pisa.tree_attention(s, cache, q, dk, dv, tmask(mask), i32(lens), ws)
    rest = [t for t in range(T) if t not in (2, 3, T - 1)]
    assert (host(O)[:, :, rest] - host(clean)[:, :, rest]).__abs__().max() <= 2.0 ** -7 * np.abs(host(clean)).max()
    assert torch.equal(l[:, :, rest], lc[:, :, rest])
    assert bool(torch.isnan(O[:, :, [2, T - 1]]).all()) and bool(torch.isinf(O[:, :, 3]).all())


def test_cached_rows_that_are_not_finite_make_nan(pisa):
    """A cached row with a NaN (exponent 255) makes every token that attends it NaN, and no other sequence."""
    import torch
    case = (2, 2, 1, 3, 128, 128, 1, 64, 0, 0, 0, [100, 100], "chain")
    s, cache, k, v, q, dk, dv, mask, lens, idx = tree_inputs(pisa, case, 24)
    ws = pisa.new_tree_workspace(s, "cuda")
    a, _ = pisa.tree_attention(s, cache, q, dk, dv, tmask(mask), i32(lens), ws)
    sws = pisa.new_cache_workspace("cuda")
    rk, rv = pisa.cache_read(cache, 1, sws, start=i32([17, 17]))
    for name in ("K", "V"):
        rows = dict(K=rk.clone(), V=rv.clone())
        rows[name][1, 0, 0, 5] = float("nan") if name == "K" else float("inf")
        pisa.cache_write(cache, rows["K"], rows["V"], sws, start=i32([17, 17]), count=i32([0, 1]))
        b, l = pisa.tree_attention(s, cache, q, dk, dv, tmask(mask), i32(lens), ws)
        assert torch.equal(a[0], b[0]) and bool(torch.isnan(b[1]).all())
        assert bool(torch.isnan(l[1]).all()) == (name == "K")
        pisa.cache_write(cache, rk, rv, sws, start=i32([17, 17]), count=i32([0, 1]))
    c, _ = pisa.tree_attention(s, cache, q, dk, dv, tmask(mask), i32(lens), ws)
    assert torch.equal(a, c)


@pytest.mark.parametrize("fmt", [0, 1])
def test_tree_bad_indices_and_lengths_are_recorded(pisa, fmt):
    import torch
    case = (3, 4, 2, 2, 512, 64, fmt, 64, 384, 4, 0, [400, 384, 10], "chain")
    s, cache, k, v, q, dk, dv, mask, lens, idx = tree_inputs(pisa, case, 25)
    ws = pisa.new_tree_workspace(s, "cuda")
    good, gl = pisa.tree_attention(s, cache, q, dk, dv, tmask(mask), i32(lens), ws, idx=i32(idx))
    assert pisa.check_status(ws) == (pisa.OK, 0)
    bad = idx.copy()
    short = np.argwhere(idx[:, :, 0, -1] < 0)[0]
    bad[short[0], short[1], 0, -1] = 6                                   # block 6 of 0..5
    O, l = pisa.tree_attention(s, cache, q, dk, dv, tmask(mask), i32(lens), ws, idx=i32(bad))
    st, detail = pisa.check_status(ws)
    assert (st, detail) == (pisa.ERR_BAD_INDEX, 0x7B1)
    assert torch.equal(O, good) and torch.equal(l, gl)                   # the entry is skipped
    for wrong, same in (([400, 384, -5], [400, 384, 0]), ([4000, 384, 10], [512, 384, 10])):
        O, l = pisa.tree_attention(s, cache, q, dk, dv, tmask(mask), i32(wrong), ws, idx=i32(idx))
        assert pisa.check_status(ws) == (pisa.ERR_BAD_INDEX, 0x7B0)
        if same[0] == 400:
            O2, l2 = pisa.tree_attention(s, cache, q, dk, dv, tmask(mask), i32(same), ws, idx=i32(idx))
            assert torch.equal(O, O2) and torch.equal(l, l2)


def test_tree_repeated_blocks_count_twice(pisa):
    case = (1, 2, 1, 2, 256, 128, 1, 64, 192, 3, 0, [200], "chain")
    s, cache, k, v, q, dk, dv, mask, lens, idx = tree_inputs(pisa, case, 26)
    idx[:] = [1, 1, 2]
    ws = pisa.new_tree_workspace(s, "cuda")
    O, lse = pisa.tree_attention(s, cache, q, dk, dv, tmask(mask), i32(lens), ws, idx=i32(idx))
    check_tree(s, O, lse, k, v, q, dk, dv, mask, lens, idx)


def test_tree_matches_the_decode_step(pisa):
    """One token that attends no drafted token, over a bf16 cache and the blocks that pisa_select_blocks
    chose, is the library's decode attention."""
    import torch
    rng = np.random.default_rng(27)
    B, Hq, Hkv, cap, D, topk = 3, 8, 2, 2048, 128, 9
    cache, k, v = fill(pisa, rng, pisa.CacheShape(B, Hkv, cap, D, pisa.CACHE_BF16))
    q = bf16(rng, B, Hq, 1, D)
    shape = pisa.Shape(B, Hq, Hkv, 1, 1920, D, 64, 4, topk, kv_capacity=cap)
    ws0 = pisa.new_workspace(shape, "cuda")
    idx = pisa.select_blocks(shape, q, pisa.build_pyramid(shape, cache.k), ws0)
    O0, l0 = pisa.sparse_attention(shape, q, cache.k, cache.v, idx, ws0)
    s = pisa.TreeShape(B, Hq, Hkv, 1, cap, D, pisa.CACHE_BF16, 64, 1920, topk)
    ws = pisa.new_tree_workspace(s, "cuda")
    none = torch.zeros((B, 1), dtype=torch.int64, device="cuda")
    d = torch.full((B, Hkv, 1, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    O, l = pisa.tree_attention(s, cache, q, d, d, none, i32([1920] * B), ws, idx=idx)
    assert np.abs(host(O) - host(O0)).max() <= 2.0 ** -7 * np.abs(host(O0)).max()
    assert np.abs(host(l) - host(l0)).max() <= 2.0 ** -16 * 16


def test_tree_refusals(pisa):
    import torch
    case = (2, 4, 2, 3, 256, 64, 1, 64, 192, 2, 0, [200, 192], "chain")
    s, cache, k, v, q, dk, dv, mask, lens, idx = tree_inputs(pisa, case, 28)
    ws = pisa.new_tree_workspace(s, "cuda")
    ok = dict(Q=q, K=dk, V=dv, mask=tmask(mask), cache_len=i32(lens), ws=ws, idx=i32(idx))
    for bad in (dict(Q=q.float()), dict(Q=q[:, :, :2]), dict(K=q), dict(V=dv.transpose(2, 3)), dict(mask=tmask(mask).int()),
                dict(mask=tmask(mask)[:1]), dict(cache_len=i32([1])), dict(cache_len=i32(lens).long()), dict(idx=None),
                dict(idx=i32(idx)[..., :1]), dict(ws=ws[:-1]), dict(ws=ws.cpu()), dict(mask=tmask(mask).cpu()),
                dict(O=q.float()), dict(lse=q)):
        with pytest.raises((ValueError, pisa.PisaError)):
            pisa.tree_attention(s, cache, **{**ok, **bad})
    with pytest.raises(ValueError):
        pisa.tree_attention(dataclasses.replace(s, format=0), cache, **ok)
    with pytest.raises(ValueError):
        pisa.tree_attention(dataclasses.replace(s, capacity=512), cache, **ok)


# ----------------------------------------------------------------------------- streams, graphs

def test_other_stream_and_graph(pisa):
    """The calls run on the stream they are given and can be captured; a replay sees new inputs and
    lengths, and the eager results of the same inputs come back bit for bit."""
    import torch
    case = (3, 8, 2, 5, 1024, 128, 1, 64, 896, 4, 0, [1000, 900, 20], "tree")
    s, cache, k, v, q, dk, dv, mask, lens, idx = tree_inputs(pisa, case, 31)
    ws = pisa.new_tree_workspace(s, "cuda")
    m, n, ix = tmask(mask), i32(lens), i32(idx)
    nr = pisa.NormRopeShape(3, 5, 8, 2, 128, 128)
    rng = np.random.default_rng(32)
    x = bf16(rng, 3, 5, 12, 128)
    pos, fr, w = i32(lens[:, None] + np.arange(5)), f32(10000.0 ** (-np.arange(64) / 64)), f32(np.ones(128))
    Q, K = torch.empty_like(q), torch.empty_like(dk)
    O, lse = torch.empty_like(q), torch.empty((3, 8, 5), device="cuda")
    cnt = i32([1, 2, 5])

    def step(stream=None):
        pisa.qk_norm_rope(nr, x[:, :, :8], x[:, :, 8:10], pos, fr, w, w, Q=Q, K=K, stream=stream)
        pisa.tree_attention(s, cache, Q, K, dv, m, n, ws, idx=ix, O=O, lse=lse, stream=stream)
        pisa.cache_write(cache, K, dv, ws, start=n, count=cnt, stream=stream)

    snap = raw(cache)

    def restore():
        for t, y in zip((cache.k, cache.v, cache.k_exp, cache.v_exp), snap):
            t.view(torch.uint8).copy_(torch.from_numpy(y))

    step()
    want = (O.clone(), lse.clone(), raw(cache))
    restore()
    O.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(O, want[0]) and torch.equal(lse, want[1])
    restore()
    O.zero_()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        restore()
        O.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(O, want[0]) and torch.equal(lse, want[1])
        assert all(np.array_equal(a, b) for a, b in zip(raw(cache), want[2]))
    # other lengths (shorter: what lies past the old ones is NaN), the same graph
    restore()
    n.copy_(i32([950, 0, 10]))
    graph.replay()
    got = O.clone()
    restore()
    step()
    assert torch.equal(O, got)
    assert pisa.check_status(ws) == (pisa.OK, 0)


# ----------------------------------------------------------------------------- together

@pytest.mark.parametrize("fmt, T, Hq, D", [(1, 2, 8, 128), (1, 12, 4, 128), (1, 20, 8, 64), (0, 48, 8, 128)])
def test_two_calls_at_once(pisa, fmt, T, Hq, D):
    """Calls with a workspace each, on two streams and in two graphs that run at the same time, keep their bits."""
    import torch
    case = (6, Hq, 2, T, 2048, D, fmt, 64, 0, 0, 0, [2000, 1, 1500, 0, 777, 2048], "tree")
    s, cache, k, v, q, dk, dv, mask, lens, idx = tree_inputs(pisa, case, 41)
    m, n, q2 = tmask(mask), i32(lens), (q.float() * 0.5).to(torch.bfloat16)
    ws = [pisa.new_tree_workspace(s, "cuda") for _ in range(2)]
    want = [pisa.tree_attention(s, cache, x, dk, dv, m, n, ws[0])[0].clone() for x in (q, q2)]
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(q) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(8):
        for i, x in enumerate((q, q2)):
            pisa.tree_attention(s, cache, x, dk, dv, m, n, ws[i], O=outs[i], lse=False, stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graphs = []
    for i, x in enumerate((q, q2)):
        outs[i].zero_()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            pisa.tree_attention(s, cache, x, dk, dv, m, n, ws[i], O=outs[i], lse=False)
    for _ in range(8):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert [pisa.check_status(w) for w in ws] == [(pisa.OK, 0)] * 2


@pytest.mark.parametrize("fmt, T", [(1, 1), (1, 20), (0, 2), (0, 20)])
def test_offsets_past_32_bits(pisa, fmt, T):
    """The end of a cache whose last rows lie past 2^32 bytes gives the bits of a small cache of the same rows."""
    import torch
    rng = np.random.default_rng(42)
    D, H, rows = 128, 3, 2 ** (24 if fmt else 23)
    k, v, q, dk, dv = (bf16(rng, 1, h, n, D) for h, n in ((H, 190), (H, 190), (2 * H, T), (H, T), (H, T)))
    m = tmask(tree_bits(rng, 1, T, "chain"))
    got = []
    for cap in (192, rows):
        cs = pisa.CacheShape(1, H, cap, D, fmt)
        dt = torch.float8_e4m3fn if fmt else torch.bfloat16
        kv = [torch.empty((1, H, cap, D), dtype=dt, device="cuda") for _ in range(2)]
        ex = [torch.empty((1, H, cap), dtype=torch.uint8, device="cuda") if fmt else None for _ in range(2)]
        cache = pisa.Cache(cs, *kv, *ex)
        ws = pisa.new_cache_workspace("cuda")
        pisa.cache_write(cache, k, v, ws, start=i32([cap - 192]))
        back = pisa.cache_read(cache, 190, ws, start=i32([cap - 192]))
        s = pisa.TreeShape(1, 2 * H, H, T, cap, D, fmt, 64, cap - 64, 2)
        tw = pisa.new_tree_workspace(s, "cuda")
        idx = torch.tensor([cap // 64 - 3, cap // 64 - 2], dtype=torch.int32, device="cuda").repeat(1, H, 1, 1)
        O, lse = pisa.tree_attention(s, cache, q, dk, dv, m, i32([cap - 2]), tw, idx=idx)
        assert pisa.check_status(ws) == (pisa.OK, 0) and pisa.check_status(tw) == (pisa.OK, 0)
        got.append((*back, O, lse))
        del cache, kv, ex
    assert all(torch.equal(a, b) for a, b in zip(*got))
    torch.cuda.empty_cache()


def test_serving_loop(pisa):
    """Prompt into the cache, pyramid, then steps of: norm and rotation of five drafted tokens, selection
    for the first, tree attention over the 8-bit cache, two accepted tokens written, pyramid appended as
    blocks fill. Every step's output is checked against the oracle on the cache's own values."""
    import torch
    rng = np.random.default_rng(41)
    B, Hq, Hkv, D, T, blk, topk, cap = 2, 4, 2, 128, 5, 64, 3, 640
    cs = pisa.CacheShape(B, Hkv, cap, D)
    cache = pisa.new_cache(cs, "cuda")
    w, fr = 1 + 0.2 * rng.standard_normal(D), (10000.0 ** (-np.arange(64) / 64)).astype(np.float32)
    tw, tf = f32(w), f32(fr)
    sws = pisa.new_cache_workspace("cuda")

    def project(t, pos):
        x = bf16(rng, B, t, Hq + 2 * Hkv, D)
        Q, K = pisa.qk_norm_rope(pisa.NormRopeShape(B, t, Hq, Hkv, D, D), x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], i32(pos), tf, tw, tw)
        return x, Q, K, x[:, :, Hq + Hkv:].transpose(1, 2)

    lens = np.array([330, 318])
    _, _, K, V = project(330, np.tile(np.arange(330), (B, 1)))
    pisa.cache_write(cache, K, V, sws, count=i32(lens))
    covered, pyr = 0, None
    mask = tree_bits(rng, B, T, "tree")
    for step in range(40):
        full = int(lens.min()) // blk * blk                              # blocks that every sequence has filled
        shape = pisa.Shape(B, Hq, Hkv, 1, full, D, blk, 4, topk, kv_capacity=cap)
        if pyr is None:
            pyr = torch.zeros((B, Hkv, shape.n_nodes, D), device="cuda")
        pisa.cache_append_pyramid(shape, cache, pyr, covered)
        covered = full
        x, Q, K, V = project(T, lens[:, None] + np.arange(T))
        V = V.contiguous()
        ws0 = pisa.new_workspace(shape, "cuda")
        idx = pisa.select_blocks(shape, Q[:, :, :1].contiguous(), pyr, ws0)
        s = pisa.TreeShape(B, Hq, Hkv, T, cap, D, cs.format, blk, full, topk)
        ws = pisa.new_tree_workspace(s, "cuda")
        O, lse = pisa.tree_attention(s, cache, Q, K, V, tmask(mask), i32(lens), ws, idx=idx)
        assert pisa.check_status(ws) == (pisa.OK, 0) and pisa.check_status(ws0) == (pisa.OK, 0)
        if step % 8 == 0:
            k, v, ke, ve = raw(cache)
            check_tree(s, O, lse, so.row_values(k, ke), so.row_values(v, ve), Q, K, V, mask, lens, idx.cpu().numpy(), step)
            assert bool((idx >= 0).sum() == B * Hkv * min(topk, full // blk))
        count = np.array([2, 1 + step % 3])
        pisa.cache_write(cache, K, V, sws, start=i32(lens), count=i32(count))
        lens = lens + count
    assert pisa.check_status(sws) == (pisa.OK, 0) and covered == 384
    again = torch.zeros_like(pyr)
    pisa.cache_append_pyramid(dataclasses.replace(shape, seq_kv=covered), cache, again, 0)
    assert torch.equal(again, pyr)


def test_training_step(pisa):
    """Projection -> norm and rotation -> sparse attention, forward and backward, into a packed gradient:
    the gradient of the whole against differences of the fp64 loss through a fixed selection."""
    import torch
    rng = np.random.default_rng(42)
    B, N, Hq, Hkv, D, blk, topk = 1, 256, 4, 2, 64, 64, 2
    x = bf16(rng, B, N, Hq + 2 * Hkv, D)
    wq, wk = (1 + 0.2 * rng.standard_normal(D)).astype(np.float32), (1 + 0.2 * rng.standard_normal(D)).astype(np.float32)
    pos, fr = np.arange(N)[None].astype(np.int32), (100.0 ** (-np.arange(16) / 16)).astype(np.float32)
    nr = pisa.NormRopeShape(B, N, Hq, Hkv, D, 32)
    shape = pisa.Shape(B, Hq, Hkv, N, N, D, blk, 4, topk, causal=1)
    ws = pisa.new_workspace(shape, "cuda")
    args = (i32(pos), f32(fr))
    Q, K = pisa.qk_norm_rope(nr, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], *args, f32(wq), f32(wk))
    V = x[:, :, Hq + Hkv:].transpose(1, 2).contiguous()
    O, lse, idx = pisa.forward(shape, Q, K, V, ws, idx=True)
    dO = bf16(rng, B, Hq, N, D)
    dQ, dK, dV = pisa.sparse_attention_backward(shape, Q, K, V, O, lse, dO, idx)
    grad = torch.empty_like(x)
    _, _, dwq, dwk = pisa.qk_norm_rope_backward(nr, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], *args, dQ, dK, f32(wq), f32(wk),
                                                dXq=grad[:, :, :Hq], dXk=grad[:, :, Hq:Hq + Hkv])
    grad[:, :, Hq + Hkv:] = dV.transpose(1, 2)
    sel, g, xh, doh = idx.cpu().numpy(), Hq // Hkv, host(x), host(dO)

    def loss(xx, a, b):
        q = so.norm_rope(xx[:, :, :Hq], a, pos, fr, 32, False, 1e-6)
        k = so.norm_rope(xx[:, :, Hq:Hq + Hkv], b, pos, fr, 32, False, 1e-6)
        v = xx[:, :, Hq + Hkv:].transpose(0, 2, 1, 3)
        total = 0.0
        for h in range(Hq):
            for i in range(N // blk):
                at = np.concatenate([np.arange(j * blk, (j + 1) * blk) for j in sel[0, h // g, i] if j >= 0])
                rows = np.arange(i * blk, (i + 1) * blk)
                s = q[0, h, rows] @ k[0, h // g, at].T / math.sqrt(D)
                s[at[None] > rows[:, None]] = -np.inf
                p = np.exp(s - s.max(-1, keepdims=True))
                total += ((p @ v[0, h // g, at] / p.sum(-1, keepdims=True)) * doh[0, h, rows]).sum()
        return total

    h = 1e-5
    for t in range(4):
        u = rng.standard_normal(xh.shape)
        a, b = rng.standard_normal(D), rng.standard_normal(D)
        num = (loss(xh + h * u, wq + h * a, wk + h * b) - loss(xh - h * u, wq - h * a, wk - h * b)) / (2 * h)
        parts = (host(grad) * u, host(dwq) * a, host(dwk) * b)
        got = sum(p.sum() for p in parts)
        # bf16 dQ, dK, dV, O and grad: five roundings of 2^-8 and bf16 P and dS, random in sign over the
        # terms: 8 roundings of 2^-8 of the terms' root sum of squares, six deviations wide
        tol = 6 * 8 * 2.0 ** -8 * math.sqrt(sum((p ** 2).sum() for p in parts))
        assert abs(num - got) <= tol, (num, got, tol)
