"""CPU oracle of the operators around the attention, in numpy fp64: norm and rotation of queries and
keys with their gradient, the e4m3 cache's rows, and the attention of drafted tokens over a cache.

Written from the formulas of include/pisa.h; it shares no code with the CUDA side.
"""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0


# ----------------------------------------------------------------------------- norm and rotation

def _pair_axes(R: int, interleaved: bool):
    i = np.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def rotate(u, pos, inv_freq, R, interleaved, sign=1.0):
    """u [B, T, H, D] turned by pos [B, T] * inv_freq [R/2]; sign -1 turns back."""
    y = np.array(u, dtype=np.float64)
    if R == 0:
        return y
    t = np.asarray(pos, np.float64)[:, :, None, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(t), sign * np.sin(t)
    a, b = _pair_axes(R, interleaved)
    y[..., a] = u[..., a] * c - u[..., b] * s
    y[..., b] = u[..., a] * s + u[..., b] * c
    return y


def norm_rope(x, w, pos, inv_freq, R, interleaved, eps):
    """x [B, T, H, D] -> [B, H, T, D]."""
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = x * r * (1.0 if w is None else np.asarray(w, np.float64))
    return rotate(u, pos, inv_freq, R, interleaved).transpose(0, 2, 1, 3)


def norm_rope_backward(x, w, pos, inv_freq, R, interleaved, eps, dy):
    """dy [B, H, T, D] -> dx [B, T, H, D], dw [D], and the size that dw's rounding errors go by: a term is
    (c dy_a + s dy_b) x r, whose two products may cancel, so its error is relative to
    (|dy_a| + |dy_b|) |x r| (|c|, |s| <= 1) and not to the term."""
    x = np.asarray(x, np.float64)
    D = x.shape[-1]
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    du = rotate(np.asarray(dy, np.float64).transpose(0, 2, 1, 3), pos, inv_freq, R, interleaved, -1.0)
    dn = du * (1.0 if w is None else np.asarray(w, np.float64))
    dx = r * dn - r ** 3 * x * (dn * x).sum(-1, keepdims=True) / D
    size = np.abs(np.asarray(dy, np.float64)).transpose(0, 2, 1, 3)
    both = size.copy()
    a, b = _pair_axes(R, interleaved)
    both[..., a] = both[..., b] = size[..., a] + size[..., b]
    return dx, (du * x * r).sum((0, 1, 2)), (both * np.abs(x) * r).sum((0, 1, 2))


# ----------------------------------------------------------------------------- e4m3 rows

def e4m3_grid() -> np.ndarray:
    """The 127 non-negative finite values, by byte."""
    out = []
    for byte in range(127):
        e, m = byte >> 3, byte & 7
        out.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(out)


def round_e4m3(v):
    """Bytes of the nearest e4m3 values (ties to the even byte), |v| <= 448."""
    grid = e4m3_grid()
    a = np.abs(v)
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    byte = np.where(up, hi, lo).astype(np.uint8)
    return byte | (np.signbit(v).astype(np.uint8) << 7)


def quantise_rows(x):
    """x [..., D] -> (bytes [..., D], exponent bytes [...])."""
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x).all(-1)
    top = np.abs(np.where(np.isfinite(x), x, 0.0)).max(-1)
    e = np.full(top.shape, 1, np.int64)
    for byte in range(1, 255):
        e[top > E4M3_MAX * 2.0 ** (byte - 127)] = byte + 1
    q = round_e4m3(np.where(bad[..., None], 0.0, np.where(np.isfinite(x), x, 0.0) * 2.0 ** (127.0 - e[..., None])))
    q[bad] = 0
    e[bad] = 255
    return q, e.astype(np.uint8)


def row_values(q, e):
    """Values of e4m3 bytes with exponent bytes (byte 255: NaN)."""
    grid = np.concatenate([e4m3_grid(), [np.nan]])
    v = grid[q & 0x7F] * np.where(q & 0x80, -1.0, 1.0)
    scale = np.where(e == 255, np.nan, 2.0 ** (e.astype(np.float64) - 127))
    return v * scale[..., None]


# ----------------------------------------------------------------------------- drafted tokens

def seen_positions(length, cap, seq_kv, topk, block, idx_row):
    """Cache positions that a selection row lets its tokens attend, in order (repeats kept)."""
    length = min(max(int(length), 0), cap)
    if topk == 0:
        return np.arange(length)
    at = [np.arange(j * block, (j + 1) * block) for j in idx_row if 0 <= j < seq_kv // block]
    at.append(np.arange(seq_kv, max(seq_kv, length)))
    at = np.concatenate(at)
    return at[at < length]


def tree_attention(q, dk, dv, mask, k, v, length, idx, *, block, seq_kv, topk, per_qhead, scale):
    """q [B, Hq, T, D], drafted dk, dv [B, Hkv, T, D], mask [B, T] (int), cache values k, v
    [B, Hkv, cap, D], all fp64. Returns O, LSE and, for tolerances, sum_j p_j |v_j| and the largest
    sum_i |q_i k_ij| of each row."""
    B, Hq, T, D = q.shape
    Hkv, cap = k.shape[1], k.shape[2]
    g = Hq // Hkv
    scale = scale if scale > 0 else 1.0 / math.sqrt(D)
    O, A = np.zeros((B, Hq, T, D)), np.zeros((B, Hq, T, D))
    L, S = np.full((B, Hq, T), -np.inf), np.zeros((B, Hq, T))
    for b in range(B):
        for h in range(Hq):
            kv = h // g
            row = idx[b, h if per_qhead else kv, 0] if topk else None
            at = seen_positions(length[b], cap, seq_kv, topk, block, row)
            for t in range(T):
                js = [j for j in range(T) if (int(mask[b, t]) >> j) & 1]
                kk = np.concatenate([k[b, kv][at], dk[b, kv][js]])
                vv = np.concatenate([v[b, kv][at], dv[b, kv][js]])
                if len(kk) == 0:
                    continue
                s = (kk @ q[b, h, t]) * scale
                m = s.max()
                p = np.exp(s - m)
                O[b, h, t] = p @ vv / p.sum()
                L[b, h, t] = m + math.log(p.sum()) if np.isfinite(m) else np.nan
                A[b, h, t] = p @ np.abs(vv) / p.sum()
                S[b, h, t] = (np.abs(kk) @ np.abs(q[b, h, t])).max() * scale
    return O, L, A, S
