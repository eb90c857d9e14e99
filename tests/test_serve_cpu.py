"""Argument checks of the calls around the attention, and pins of their oracle. No GPU: every compute
call here fails validation on the host, so the fake pointers are never handed to a kernel."""
import ctypes
import math

import numpy as np
import pytest

from oracle import serve_oracle as so

pisa = pytest.importorskip("block_sparse_long_pisa_b200")
FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)
ODD4 = ctypes.c_void_p((1 << 20) + 2)
BIG = 1 << 40
f = pisa._lib


# ----------------------------------------------------------------------------- norm and rotation

def nr(**kw):
    a = dict(batch=2, tokens=3, heads_q=4, heads_kv=2, head_dim=64, rotary_dim=64, interleaved=0, eps=1e-6)
    strides = {k: kw.pop(k) for k in ("xq", "xk", "dxq", "dxk") if k in kw}
    a.update(kw)
    d = 64
    st = dict(xq=(3 * 4 * d, 4 * d, d), xk=(3 * 2 * d, 2 * d, d), dxq=(3 * 4 * d, 4 * d, d), dxk=(3 * 2 * d, 2 * d, d))
    st.update(strides)
    return pisa.NormRopeShape(**a).c(*[st[k] for k in ("xq", "xk", "dxq", "dxk")])


@pytest.mark.parametrize("bad, code", [
    (dict(batch=0), 1), (dict(tokens=0), 1), (dict(heads_q=0), 1), (dict(heads_kv=-1), 1), (dict(rotary_dim=-16), 1),
    (dict(rotary_dim=80), 1), (dict(interleaved=2), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1), (dict(xq=(768, 256, 60)), 1), (dict(xk=(384, -128, 64)), 1), (dict(head_dim=96), 2),
    (dict(rotary_dim=24), 2), (dict(batch=1 << 16, tokens=1 << 16), 2),
])
def test_norm_rope_refuses_shapes(bad, code):
    s = nr(**bad)
    assert f.pisa_qk_norm_rope(s, FAKE, FAKE, None, None, FAKE, FAKE, FAKE, FAKE, None) == code
    assert f.pisa_qk_norm_rope_backward(s, FAKE, FAKE, None, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, FAKE,
                                        BIG, None) == code
    n = ctypes.c_size_t()
    assert f.pisa_norm_rope_workspace_size(s, n) == code


def test_norm_rope_refuses_pointers():
    s = nr()
    args = [FAKE, FAKE, None, None, FAKE, FAKE, FAKE, FAKE]
    for i in (0, 1, 6, 7):
        for p in (None, ODD):
            a = list(args)
            a[i] = p
            assert f.pisa_qk_norm_rope(s, *a, None) == pisa.ERR_INVALID_ARG
    for i in (4, 5):
        a = list(args)
        a[i] = None
        assert f.pisa_qk_norm_rope(s, *a, None) == pisa.ERR_INVALID_ARG
    for i in (2, 3, 4, 5):
        a = list(args)
        a[i] = ODD4
        assert f.pisa_qk_norm_rope(s, *a, None) == pisa.ERR_INVALID_ARG
    assert f.pisa_qk_norm_rope(None, *args, None) == pisa.ERR_INVALID_ARG


def test_norm_rope_backward_refuses():
    s = nr()
    need = pisa.norm_rope_workspace_size(pisa.NormRopeShape(2, 3, 4, 2, 64, 64))
    args = [FAKE, FAKE, None, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, FAKE]
    assert f.pisa_qk_norm_rope_backward(s, *args, need - 1, None) == pisa.ERR_WORKSPACE
    for i in (0, 1, 6, 7, 8, 9, 12):
        for p in (None, ODD):
            a = list(args)
            a[i] = p
            assert f.pisa_qk_norm_rope_backward(s, *a, need, None) == pisa.ERR_INVALID_ARG
    for i in (10, 11):
        a = list(args)
        a[i] = ODD4
        assert f.pisa_qk_norm_rope_backward(s, *a, need, None) == pisa.ERR_INVALID_ARG


@pytest.mark.parametrize("dxq, ok", [
    ((768, 256, 64), True), ((0, 256, 64), False), ((768, 0, 64), False), ((768, 256, 0), False),
    ((768, 256, 56), False), ((256, 512, 64), True), ((64 * 8 * 3, 64 * 8, 64), True), ((64, 128, 384), True),
    ((704, 256, 64), False), ((64, 64, 64), False), ((1 << 62, 256, 64), False),
])
def test_norm_rope_backward_refuses_overlapping_gradients(dxq, ok, monkeypatch):
    monkeypatch.setenv("PISA_FAULT", "launch")   # a call that passes its checks ends in ERR_CUDA
    args = [FAKE, FAKE, None, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, BIG, None]
    assert f.pisa_qk_norm_rope_backward(nr(dxq=dxq), *args) == (pisa.ERR_CUDA if ok else pisa.ERR_INVALID_ARG)


# ----------------------------------------------------------------------------- the cache

@pytest.mark.parametrize("bad, code", [
    (dict(batch=0), 1), (dict(heads_kv=0), 1), (dict(capacity=0), 1), (dict(format=2), 1), (dict(head_dim=32), 2),
    (dict(batch=1 << 15, capacity=1 << 16), 2),
])
def test_cache_refuses_shapes(bad, code):
    a = dict(batch=2, heads_kv=2, capacity=64, head_dim=64, format=pisa.CACHE_E4M3)
    a.update(bad)
    s = pisa.CacheShape(**a).c()
    st = (ctypes.c_int64 * 3)(128, 64, 64)
    assert f.pisa_cache_write(s, 1, FAKE, FAKE, st, st, None, None, FAKE, FAKE, FAKE, FAKE, FAKE, None) == code
    assert f.pisa_cache_read(s, 1, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, FAKE, FAKE, None) == code


def test_cache_refuses_arguments():
    s = pisa.CacheShape(2, 2, 64, 64, pisa.CACHE_E4M3).c()
    plain = pisa.CacheShape(2, 2, 64, 64, pisa.CACHE_BF16).c()
    st = (ctypes.c_int64 * 3)(128, 64, 64)
    good = [s, 1, FAKE, FAKE, st, st, None, None, FAKE, FAKE, FAKE, FAKE, FAKE]

    def write(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f.pisa_cache_write(*a, None)

    for tokens in (0, -1, 65):
        assert write(_1=tokens) == pisa.ERR_INVALID_ARG
    for i in (2, 3, 8, 9, 12):
        assert write(**{f"_{i}": None}) == pisa.ERR_INVALID_ARG
        assert write(**{f"_{i}": ODD}) == pisa.ERR_INVALID_ARG
    for i in (10, 11):
        assert write(**{f"_{i}": None}) == pisa.ERR_INVALID_ARG       # e4m3 without exponents
    assert write(_0=plain) == pisa.ERR_INVALID_ARG                    # bf16 with them
    for i in (6, 7):
        assert write(**{f"_{i}": ODD4}) == pisa.ERR_INVALID_ARG
    for bad in ((128, 64, 60), (128, -64, 64)):
        assert write(_4=(ctypes.c_int64 * 3)(*bad)) == pisa.ERR_INVALID_ARG
        assert write(_5=(ctypes.c_int64 * 3)(*bad)) == pisa.ERR_INVALID_ARG
    read = [s, 1, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, FAKE, FAKE]
    for i in (2, 3, 4, 5, 8, 9, 10):
        a = list(read)
        a[i] = None
        assert f.pisa_cache_read(*a, None) == pisa.ERR_INVALID_ARG
    for tokens in (0, 65):
        assert f.pisa_cache_read(s, tokens, *read[2:], None) == pisa.ERR_INVALID_ARG


def test_cache_append_pyramid_refuses():
    s = pisa.Shape(2, 2, 2, 1, 256, 64, 64, 4, 1, kv_capacity=512).c()
    assert f.pisa_cache_append_pyramid(s, None, FAKE, FAKE, 0, None) == pisa.ERR_INVALID_ARG
    assert f.pisa_cache_append_pyramid(s, FAKE, None, FAKE, 0, None) == pisa.ERR_INVALID_ARG
    assert f.pisa_cache_append_pyramid(s, FAKE, FAKE, ODD, 0, None) == pisa.ERR_INVALID_ARG
    for old in (-64, 320, 32):
        assert f.pisa_cache_append_pyramid(s, FAKE, FAKE, FAKE, old, None) == pisa.ERR_INVALID_ARG


# ----------------------------------------------------------------------------- drafted tokens

TREE = dict(batch=2, heads_q=4, heads_kv=2, drafts=3, capacity=256, head_dim=64, format=1, block=64, seq_kv=128, topk=2)


@pytest.mark.parametrize("bad, code", [
    (dict(batch=0), 1), (dict(heads_q=3), 1), (dict(drafts=0), 1), (dict(format=3), 1), (dict(topk=-1), 1),
    (dict(seq_kv=96), 1), (dict(seq_kv=0), 1), (dict(seq_kv=320), 1), (dict(topk=0), 1), (dict(capacity=200), 1),
    (dict(select_per_qhead=2), 1), (dict(topk=0, seq_kv=0, select_per_qhead=1), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(head_dim=96), 2), (dict(block=32), 2), (dict(drafts=65), 2),
    (dict(topk=4097), 2), (dict(batch=1 << 20, capacity=1 << 12), 2),
])
def test_tree_refuses_shapes(bad, code):
    s = pisa.TreeShape(**{**TREE, **bad}).c()
    n = ctypes.c_size_t()
    assert f.pisa_tree_workspace_size(s, n) == code
    assert f.pisa_tree_attention(s, *[FAKE] * 12, FAKE, BIG, None) == code


def test_tree_refuses_arguments():
    s = pisa.TreeShape(**TREE)
    need = pisa.tree_workspace_size(s)
    c = s.c()
    args = [FAKE] * 13
    assert f.pisa_tree_attention(c, *args, need - 1, None) == pisa.ERR_WORKSPACE
    for i in range(13):
        if i == 11:
            continue                                  # lse is optional
        a = list(args)
        a[i] = None
        assert f.pisa_tree_attention(c, *a, need, None) == pisa.ERR_INVALID_ARG, i
        a[i] = ODD4
        assert f.pisa_tree_attention(c, *a, need, None) == pisa.ERR_INVALID_ARG, i
    whole = pisa.TreeShape(**{**TREE, "topk": 0, "seq_kv": 0}).c()
    assert f.pisa_tree_attention(whole, *args, BIG, None) == pisa.ERR_INVALID_ARG      # idx without topk
    plain = pisa.TreeShape(**{**TREE, "format": 0}).c()
    assert f.pisa_tree_attention(plain, *args, BIG, None) == pisa.ERR_INVALID_ARG      # exponents of a bf16 cache


def test_injected_failure(monkeypatch):
    monkeypatch.setenv("PISA_FAULT", "launch")
    st = (ctypes.c_int64 * 3)(128, 64, 64)
    assert f.pisa_qk_norm_rope(nr(), FAKE, FAKE, None, None, FAKE, FAKE, FAKE, FAKE, None) == pisa.ERR_CUDA
    s = pisa.CacheShape(2, 2, 64, 64, pisa.CACHE_E4M3).c()
    assert f.pisa_cache_write(s, 1, FAKE, FAKE, st, st, None, None, FAKE, FAKE, FAKE, FAKE, FAKE, None) == pisa.ERR_CUDA
    assert f.pisa_tree_attention(pisa.TreeShape(**TREE).c(), *[FAKE] * 13, BIG, None) == pisa.ERR_CUDA
    assert pisa.last_launch_count() == 0


def test_workspace_sizes_depend_on_the_shape_alone():
    """Status word, then two partial slots (o, m, l of a row tile) for each of the runs."""
    for drafts, rm, runs in ((1, 8, 444), (4, 8, 444), (5, 16, 296), (8, 16, 296), (16, 16, 296), (17, 128, 148), (64, 128, 148)):
        s = pisa.TreeShape(**{**TREE, "drafts": drafts})
        assert pisa.tree_workspace_size(s) == 256 + 2 * runs * rm * 66 * 4
    assert pisa.norm_rope_workspace_size(pisa.NormRopeShape(2, 3, 4, 2, 64, 64)) == 592 * 64 * 4


# ----------------------------------------------------------------------------- pins of the oracle

def test_oracle_e4m3_grid_and_rounding():
    g = so.e4m3_grid()
    assert g[0] == 0 and g[1] == 2.0 ** -9 and g[8] == 2.0 ** -6 and g[56] == 1.0 and g[126] == 448.0
    assert np.all(np.diff(g) > 0)
    assert np.array_equal(so.round_e4m3(g), np.arange(127))
    mid = (g[1:] + g[:-1]) / 2
    assert np.all(so.round_e4m3(mid) % 2 == 0)                       # ties to even
    assert np.array_equal(so.round_e4m3(mid * (1 + 1e-9)), np.arange(1, 127))


def test_oracle_quantise_is_the_smallest_scale():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 64)) * 2.0 ** rng.integers(-40, 40, (200, 1))
    x[3] = 0
    x[4, 5] = np.inf
    x[5, 6] = np.nan
    q, e = so.quantise_rows(x)
    top = np.abs(x).max(-1)
    ok = np.isfinite(x).all(-1) & (top > 0)
    assert np.all(top[ok] <= 448 * 2.0 ** (e[ok] - 127.0))
    assert np.all(top[ok] > 448 * 2.0 ** (e[ok] - 128.0))
    assert e[3] == 1 and e[4] == 255 and e[5] == 255 and not q[4].any() and not q[5].any()
    v = so.row_values(q, e)
    s = 2.0 ** (e[ok, None] - 127.0)
    assert np.all(np.abs(v[ok] - x[ok]) <= np.maximum(2.0 ** -4 * np.abs(x[ok]), 2.0 ** -10 * s))
    assert np.isnan(v[4]).all() and np.isnan(v[5]).all()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("R", [0, 16, 64])
def test_oracle_norm_rope_gradient_against_differences(R, inter):
    rng = np.random.default_rng(R + inter)
    x, w = rng.standard_normal((2, 3, 2, 64)), 1 + 0.3 * rng.standard_normal(64)
    pos, fr = rng.integers(0, 50, (2, 3)), 10000.0 ** (-np.arange(R // 2) / max(1, R // 2))
    dy = rng.standard_normal((2, 2, 3, 64))

    def loss(x, w):
        return (so.norm_rope(x, w, pos, fr, R, inter, 1e-3) * dy).sum()

    dx, dw, _ = so.norm_rope_backward(x, w, pos, fr, R, inter, 1e-3, dy)
    for _ in range(5):
        u, v = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
        h = 1e-6
        num = (loss(x + h * u, w + h * v) - loss(x - h * u, w - h * v)) / (2 * h)
        assert abs(num - (dx * u).sum() - (dw * v).sum()) < 1e-6 * max(1.0, abs(num)) * 10
    # rotations keep norms, and position 0 turns nothing
    y = so.norm_rope(x, None, pos, fr, R, inter, 0.0)
    assert np.allclose((y ** 2).mean(-1), 1.0)
    assert np.allclose(so.norm_rope(x, w, pos * 0, fr, R, inter, 1e-3), so.norm_rope(x, w, pos, fr, 0, inter, 1e-3))


def test_oracle_tree_equals_dense_softmax_of_the_path():
    """A chain of drafted tokens over a whole cache is causal attention over cache and drafts."""
    rng = np.random.default_rng(3)
    T, n, D = 4, 37, 64
    q, dk, dv = rng.standard_normal((1, 1, T, D)), rng.standard_normal((1, 1, T, D)), rng.standard_normal((1, 1, T, D))
    k, v = rng.standard_normal((1, 1, 64, D)), rng.standard_normal((1, 1, 64, D))
    mask = np.array([[(1 << (t + 1)) - 1 for t in range(T)]])
    O, L, _, _ = so.tree_attention(q, dk, dv, mask, k, v, [n], None, block=64, seq_kv=0, topk=0, per_qhead=False, scale=0)
    kk, vv = np.concatenate([k[0, 0, :n], dk[0, 0]]), np.concatenate([v[0, 0, :n], dv[0, 0]])
    s = q[0, 0] @ kk.T / math.sqrt(D)
    s[np.arange(T)[:, None] < np.arange(n + T)[None] - n] = -np.inf
    p = np.exp(s - s.max(-1, keepdims=True))
    assert np.allclose(O[0, 0], p @ vv / p.sum(-1, keepdims=True))
    assert np.allclose(L[0, 0], s.max(-1) + np.log(p.sum(-1)))


def test_rotation_needs_positions_and_frequencies():
    torch = pytest.importorskip("torch")
    s = pisa.NormRopeShape(1, 2, 2, 1, 64, 32)
    x, y = (torch.zeros((1, 2, h, 64), dtype=torch.bfloat16) for h in (2, 1))
    pos, fr = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(16)
    for args, name in (((None, fr), "pos"), ((pos, None), "inv_freq"), ((pos.long(), fr), "pos"),
                       ((pos, fr[:8]), "inv_freq")):
        with pytest.raises(ValueError, match=name):
            pisa.qk_norm_rope(s, x, y, *args)


def test_norm_rope_backward_needs_a_workspace_of_adjacent_bytes():
    """A workspace of one repeated byte, or every other byte of one, counts more bytes than it has."""
    torch = pytest.importorskip("torch")
    s = pisa.NormRopeShape(1, 2, 2, 1, 64, 0)
    x, y = torch.zeros((1, 2, 2, 64), dtype=torch.bfloat16), torch.zeros((1, 2, 1, 64), dtype=torch.bfloat16)
    n = pisa.norm_rope_workspace_size(s)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(n), torch.zeros(2 * n, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            pisa.qk_norm_rope_backward(s, x, y, None, None, x.transpose(1, 2).contiguous(), y.transpose(1, 2).contiguous(),
                                       ws=ws)
