"""The operators around the attention in calls that an earlier form of them answered wrongly. Tolerances are those of
test_gpu_serve.py, and for few rows over an e4m3 cache one term more, derived at `floor_of`."""
import numpy as np
import pytest

from oracle import serve_oracle as so
from tests.test_gpu_serve import bf16, check_tree, f32, fill, host, i32, raw, tmask, tree_bits, tree_inputs

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


def test_calls_on_a_forked_stream_are_captured(pisa):
    """A graph whose capture forks to another stream, the calls there making their own outputs: replays give the eager bits."""
    import torch
    case = (2, 4, 2, 5, 512, 128, 1, 64, 0, 0, 0, [500, 77], "tree")
    s, cache, k, v, q, dk, dv, mask, lens, idx = tree_inputs(pisa, case, 74)
    ws, sws, m, n, count = pisa.new_tree_workspace(s, "cuda"), pisa.new_cache_workspace("cuda"), tmask(mask), i32(lens), i32([9, 4])
    nr, w = pisa.NormRopeShape(2, 5, 4, 2, 128, 0), f32(np.ones(128))
    xq, xk = q.transpose(1, 2).contiguous(), dk.transpose(1, 2).contiguous()

    def calls(stream):
        return [*pisa.tree_attention(s, cache, q, dk, dv, m, n, ws, stream=stream),
                *pisa.cache_read(cache, 9, sws, count=count, stream=stream),
                *pisa.qk_norm_rope_backward(nr, xq, xk, None, None, q, dk, w, w, stream=stream)]

    want = calls(None)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = calls(side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in got:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert pisa.check_status(ws) == (pisa.OK, 0) and pisa.check_status(sws) == (pisa.OK, 0)


# T, Hq, D: 4, 16 and two tiles of 16 rows (few), one and two tiles of 128 (many)
FORMS = [(1, 4, 128), (1, 4, 64), (4, 4, 128), (7, 2, 64), (7, 4, 128), (24, 4, 128), (40, 4, 64)]


# ----------------------------------------------------------------------------- value rows of unlike size

def floor_of(s, q, k, dk, v_exp, dv, mask, lens, idx):
    """What few rows over an e4m3 cache may be off by beside check_tree's terms. A weight (probability times its row's
    scale) times a power of two f is held in fp16, f such that the largest weight comes to 2^3 or more, and to less than
    2^16: its step is never above 2^-24 for weights below 2^-14, so rounding is off by at most 2^-25, 2^-28 of the largest
    weight; a value is at most 448 (a drafted one, whose scale is its largest magnitude over 256, at most 2^9) scales. So
    n keys: n 2^-28 2^9 max_j p_j 2^(e_j - 127) / sum p."""
    B, Hq, T, D = q.shape
    g = Hq // k.shape[1]
    out = np.zeros((B, Hq, T))
    for b in range(B):
        for h in range(Hq):
            kv = h // g
            at = so.seen_positions(lens[b], s.capacity, s.seq_kv, s.topk, s.block,
                                   idx[b, h if s.select_per_qhead else kv, 0] if s.topk else None)
            for t in range(T):
                js = [j for j in range(T) if (int(mask[b, t]) >> j) & 1]
                x = np.concatenate([k[b, kv][at], dk[b, kv][js]]) @ q[b, h, t] / np.sqrt(D)
                if len(x) == 0:
                    continue
                scale = np.concatenate([2.0 ** (v_exp[b, kv][at].astype(float) - 127), np.abs(dv[b, kv][js]).max(-1, initial=0) / 256])
                p = np.exp(x - x.max())
                out[b, h, t] = len(x) * 2.0 ** -19 * (p * scale).max() / p.sum()
    return out


def check_with_floor(s, O, lse, cache, k, v, q, dk, dv, mask, lens, idx):
    ref, L, A, S = so.tree_attention(host(q), host(dk), host(dv), mask, k, v, lens, idx, block=s.block, seq_kv=s.seq_kv,
                                     topk=s.topk, per_qhead=bool(s.select_per_qhead), scale=s.scale)
    e = 2.0 ** -18 * S
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * e[..., None]) * A
    tol += floor_of(s, host(q), k, host(dk), cache.v_exp.cpu().numpy(), host(dv), mask, lens, idx)[..., None]
    err = np.abs(host(O) - ref)
    assert (err <= tol).all(), (np.nanmax(err - tol), np.argwhere(~(err <= tol))[:5])
    assert (np.abs(host(lse) - L) <= e + 2.0 ** -20 * np.abs(L) + 2.0 ** -18).all()


@pytest.mark.parametrize("T, Hq, D", FORMS)
@pytest.mark.parametrize("top, mixed", [(20, 0), (28, 0), (34, 0), (60, 0), (100, 0), (34, 1), (60, 1)])
def test_a_large_value_row_of_vanishing_weight_hides_no_other(pisa, T, Hq, D, top, mixed):
    """Three cached value rows are 2^top times the others and their keys 2^-(top + 26) times as likely: they add nothing, and
    the others keep their precision. Mixed: every second head and token turns to those keys instead."""
    rng = np.random.default_rng(top)
    import torch
    n, cap = 150, 192
    K, V = bf16(rng, 1, 1, n, D, scale=0.25), bf16(rng, 1, 1, n, D)
    q = bf16(rng, 1, Hq, T, D, scale=0.25)
    q[..., 0] = 8.0
    if mixed:
        q[:, 1::2, :, 0] *= -1
        q[:, :, 1::2, 0] *= -1
    K[..., 0] = 0
    for at in (3, 70, 149):
        K[0, 0, at, 0] = -float(np.log(2) * (top + 26) * np.sqrt(D) / 8)
        V[0, 0, at] = V[0, 0, at] * 2.0 ** top
    dk, dv = bf16(rng, 1, 1, T, D, scale=0.25), bf16(rng, 1, 1, T, D)
    cache = pisa.new_cache(pisa.CacheShape(1, 1, cap, D), "cuda")
    pisa.cache_write(cache, K, V, pisa.new_cache_workspace("cuda"))
    kb, vb, ke, ve = raw(cache)
    s = pisa.TreeShape(1, Hq, 1, T, cap, D)
    mask, lens, ws = tree_bits(rng, 1, T, "tree"), np.array([n]), pisa.new_tree_workspace(s, "cuda")
    O, lse = pisa.tree_attention(s, cache, q, dk, dv, tmask(mask), i32(lens), ws)
    assert pisa.check_status(ws) == (pisa.OK, 0)
    check_with_floor(s, O, lse, cache, so.row_values(kb, ke), so.row_values(vb, ve), q, dk, dv, mask, lens, None)
    assert bool(torch.isfinite(O).all())


@pytest.mark.parametrize("T, Hq, D", FORMS)
@pytest.mark.parametrize("spread, qscale", [(30, 30.0), (30, 4.0), (12, 8.0), (60, 10.0)])
def test_value_rows_of_unlike_size_under_peaked_scores(pisa, T, Hq, D, spread, qscale):
    case = (3, 2 * Hq, 2, T, 704, D, 1, 64, 576, 5, 0, [700, 300, 0], "tree")
    s, cache, k, v, q, dk, dv, mask, lens, idx = tree_inputs(pisa, case, 52, spread, qscale)
    ws = pisa.new_tree_workspace(s, "cuda")
    O, lse = pisa.tree_attention(s, cache, q, dk, dv, tmask(mask), i32(lens), ws, idx=i32(idx))
    check_with_floor(s, O, lse, cache, k, v, q, dk, dv, mask, lens, idx)


@pytest.mark.parametrize("T, Hq, D", FORMS)
@pytest.mark.parametrize("big", [0, 25, 90])
def test_drafted_values_over_a_cache_of_zero_rows(pisa, T, Hq, D, big):
    """Zero rows have the smallest exponent; drafted values of 2^big beside them come out as they are."""
    rng = np.random.default_rng(7)
    cache = pisa.new_cache(pisa.CacheShape(1, 1, 128, D), "cuda")
    s = pisa.TreeShape(1, Hq, 1, T, 128, D)
    q, dk, dv = bf16(rng, 1, Hq, T, D), bf16(rng, 1, 1, T, D), bf16(rng, 1, 1, T, D) * 2.0 ** big
    mask, lens, ws = tree_bits(rng, 1, T, "tree"), np.array([100]), pisa.new_tree_workspace(s, "cuda")
    O, lse = pisa.tree_attention(s, cache, q, dk, dv, tmask(mask), i32(lens), ws)
    zero = np.zeros((1, 1, 128, D))
    check_tree(s, O, lse, zero, zero, q, dk, dv, mask, lens, None)


# ----------------------------------------------------------------------------- scores of minus infinity

@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T, Hq, D", FORMS)
def test_keys_of_minus_infinity_come_first(pisa, T, Hq, D, fmt):
    """Two blocks of keys whose scores overflow to minus infinity, then keys with scores of about -300: the result is that
    of the later keys alone. 400 sequences of the same rows, so that a run holds several units of each."""
    rng = np.random.default_rng(9)
    import torch
    B, cap = 400, 320
    K, V = bf16(rng, 1, 1, cap, D), bf16(rng, 1, 1, cap, D)
    q = bf16(rng, 1, Hq, T, D, scale=0.05).add_(1).mul_(2.0 ** 60)
    K = (K * 0.02 - 300.0 / np.sqrt(D)) * 2.0 ** -60
    K[:, :, :128] = -2.0 ** 100
    dk, dv = bf16(rng, 1, 1, T, D), bf16(rng, 1, 1, T, D)
    wide = lambda t: t.expand(B, -1, -1, -1).contiguous()
    cache = pisa.new_cache(pisa.CacheShape(B, 1, cap, D, fmt), "cuda")
    pisa.cache_write(cache, wide(K), wide(V), pisa.new_cache_workspace("cuda"))
    if fmt:
        kb, vb, ke, ve = raw(cache)
        k, v = so.row_values(kb[:1], ke[:1]), so.row_values(vb[:1], ve[:1])
    else:
        k, v = host(cache.k[:1]), host(cache.v[:1])
    s = pisa.TreeShape(B, Hq, 1, T, cap, D, fmt, 64, 256, 4)
    idx = np.tile(np.array([0, 1, 2, 3], np.int32), (B, 1, 1, 1))
    mask, lens, ws = np.zeros((B, T), np.uint64), np.full(B, cap), pisa.new_tree_workspace(s, "cuda")
    O, lse = pisa.tree_attention(s, cache, wide(q), wide(dk), wide(dv), tmask(mask), i32(lens), ws, idx=i32(idx))
    later = np.array([-1, -1, 2, 3], np.int32).reshape(1, 1, 1, 4)
    ref, L, A, S = so.tree_attention(host(q), host(dk), host(dv), mask[:1], k, v, lens[:1], later, block=64, seq_kv=256,
                                     topk=4, per_qhead=False, scale=0.0)
    e = 2.0 ** -18 * S
    assert (np.abs(host(O) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * e[..., None]) * A).all()
    assert (np.abs(host(lse) - L) <= e + 2.0 ** -20 * np.abs(L) + 2.0 ** -18).all()


# ----------------------------------------------------------------------------- drafted tokens that are not attended

@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T, Hq, D", [(5, 1, 128), (8, 2, 64), (7, 4, 128), (24, 4, 128), (40, 4, 64)])
def test_drafts_that_are_not_attended_change_no_bit(pisa, fmt, T, Hq, D):
    """Drafted tokens 1 and 2 become other finite or non-finite rows: tokens that attend neither keep O and LSE bit for bit."""
    import torch
    case = (2, 2 * Hq, 2, T, 512, D, fmt, 64, 0, 0, 0, [500, 77], "chain")
    s, cache, k, v, q, dk, dv, mask, lens, idx = tree_inputs(pisa, case, 61)
    for t in range(T):
        mask[:, t] = np.uint64((1 << t) | (1 if t % 3 else 0b110 if t > 2 else 0))
    rest = [t for t in range(T) if t not in (1, 2) and t % 3]
    ws = pisa.new_tree_workspace(s, "cuda")
    O, lse = pisa.tree_attention(s, cache, q, dk, dv, tmask(mask), i32(lens), ws)
    for scale_k, scale_v in ((30.0, 1.0), (1.0, 2.0 ** 40), (30.0, float("inf")), (float("nan"), float("nan"))):
        dk2, dv2 = dk.clone(), dv.clone()
        dk2[:, :, 1:3] *= scale_k
        dv2[:, :, 1:3] *= scale_v
        O2, lse2 = pisa.tree_attention(s, cache, q, dk2, dv2, tmask(mask), i32(lens), ws)
        assert torch.equal(O[:, :, rest], O2[:, :, rest]) and torch.equal(lse[:, :, rest], lse2[:, :, rest])


# ----------------------------------------------------------------------------- lengths past the cache

@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T, Hq", [(2, 2), (24, 4)])
@pytest.mark.parametrize("topk", [0, 2])
def test_a_length_past_the_cache_is_its_capacity(pisa, fmt, T, Hq, topk):
    """The clamped length gives the bits of the capacity, where the cache's rows are finite up to there."""
    import torch
    case = (2, 2 * Hq, 2, T, 256, 64, fmt, 64, 192 if topk else 0, topk, 0, [256, 256], "tree")
    s, cache, k, v, q, dk, dv, mask, lens, idx = tree_inputs(pisa, case, 81)
    ws, ix = pisa.new_tree_workspace(s, "cuda"), None if idx is None else i32(idx)
    want = pisa.tree_attention(s, cache, q, dk, dv, tmask(mask), i32([256, 0]), ws, idx=ix)
    assert pisa.check_status(ws) == (pisa.OK, 0)
    for n in ([257, -1], [2147483647, -2147483648]):
        got = pisa.tree_attention(s, cache, q, dk, dv, tmask(mask), i32(n), ws, idx=ix)
        assert pisa.check_status(ws) == (pisa.ERR_BAD_INDEX, 0x7B0)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
