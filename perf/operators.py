"""Cases of the serving and training operators around the sparse attention: what is measured.

Three families, each with a plain form in elementary torch operations and the library's call:

* ``rope``  RMS norm of every query and key head and the rotation by position, in one pass, and
            its backward pass;
* ``cache`` K and V rows written into a cache of 8-bit values (or copied into a bf16 one), rows
            read back, and the key pyramid kept current from the 8-bit rows;
* ``tree``  attention of a tree of drafted tokens (one token is plain decode) over such a cache:
            the selected blocks and the tail behind them, or the whole cache.

Sizes are those of the repository's workloads (32 query / 8 KV heads of 128, contexts of 32K and
128K, 64 sequences, 64 selected blocks of 64 keys) and small or ragged ones around them.
"""
import math

import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of 64 sequences: 2,560 head rows, bound by latency
        dict(name="rope decode 64x1", kind="rope", batch=64, tokens=1, hq=32, hkv=8, dim=128, rot=128,
             interleaved=False, backward=False, weights=True, far=131072),
        # the 128K prefill of one sequence, packed projections in, attention layout out
        dict(name="rope prefill 128K", kind="rope", batch=1, tokens=131072, hq=32, hkv=8, dim=128, rot=128,
             interleaved=False, backward=False, weights=True, far=0),
        # a training step of 32K tokens, 16 heads each
        dict(name="rope backward 32K", kind="rope", batch=1, tokens=32768, hq=16, hkv=16, dim=128, rot=128,
             interleaved=False, backward=True, weights=True, far=0),
        # odd token count, small heads, partial and interleaved rotation, far positions
        dict(name="rope backward odd", kind="rope", batch=3, tokens=1537, hq=12, hkv=4, dim=64, rot=32,
             interleaved=True, backward=True, weights=True, far=1000000),
        # the new token of 64 sequences into their caches
        dict(name="cache write 64x1", kind="write", batch=64, hkv=8, tokens=1, cap=2048, dim=128, bits=8, ragged=True),
        # a 128K prompt into the cache
        dict(name="cache write 128K", kind="write", batch=1, hkv=8, tokens=131072, cap=131072, dim=128, bits=8,
             ragged=False),
        # prefixes of unlike lengths read back for a prefill that continues them
        dict(name="cache read ragged", kind="read", batch=7, hkv=8, tokens=9001, cap=16384, dim=128, bits=8,
             ragged=True),
        # the block that 64 sequences have just filled enters their pyramids
        dict(name="pyramid one block", kind="pyramid", batch=64, hkv=8, cap=16384, old=8128, new=8192, dim=128,
             block=64, factor=4),
        # the pyramids of 8 prompts of 32K keys
        dict(name="pyramid 8x32K", kind="pyramid", batch=8, hkv=8, cap=32768, old=0, new=32768, dim=128, block=64,
             factor=4),
        # small calls count latency: five drafted tokens, one short sequence, two heads of 64
        dict(name="tree 1x5 short", kind="tree", batch=1, hq=2, hkv=2, drafts=5, cap=4096, seq=0, tail=1500, dim=64,
             block=64, topk=0, per_qhead=False, bits=16, branchy=True),
        # decode over the 128K caches of 64 sequences, 64 blocks selected of 2047, tail behind them
        dict(name="tree decode 64x128K", kind="tree", batch=64, hq=32, hkv=8, drafts=1, cap=131072, seq=131008,
             tail=63, dim=128, block=64, topk=64, per_qhead=False, bits=8, branchy=False),
        # trees of 48 drafted tokens over whole bf16 caches of unlike lengths
        dict(name="tree 8x48 ragged", kind="tree", batch=8, hq=32, hkv=8, drafts=48, cap=32768, seq=0, tail=32768,
             dim=128, block=64, topk=0, per_qhead=False, bits=16, branchy=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "rope", "write", "read", "pyramid", "tree", "tree", "tree"])
    dim = rng.choice([64, 128, 128])
    if kind == "rope":
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 5, 8])
        rows = _spread(rng, 64, 32768 * 32)
        batch = rng.choice([1, 1, 2, 5, 33])
        return dict(kind=kind, batch=batch, tokens=max(1, rows // (batch * (hq + hkv))), hq=hq, hkv=hkv, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, dim // 4, dim - 16]), interleaved=rng.random() < 0.4,
                    backward=rng.random() < 0.5, weights=rng.random() < 0.8, far=rng.choice([0, 0, 5000, 1000000]))
    if kind in ("write", "read"):
        hkv = rng.choice([1, 2, 3, 8])
        batch = rng.choice([1, 2, 7, 16, 64])
        tokens = _spread(rng, 1, max(2, 400000 // (batch * hkv)))
        cap = 64 * ((tokens + 63) // 64 + rng.randrange(0, 5))
        return dict(kind=kind, batch=batch, hkv=hkv, tokens=tokens, cap=cap, dim=dim, bits=rng.choice([8, 8, 8, 16]),
                    ragged=rng.random() < 0.6)
    if kind == "pyramid":
        block = rng.choice([64, 128])
        blocks = _spread(rng, 2, 256)
        first = rng.randrange(0, blocks) if rng.random() < 0.6 else 0
        return dict(kind=kind, batch=rng.choice([1, 3, 8]), hkv=rng.choice([1, 2, 8]),
                    cap=block * (blocks + rng.randrange(0, 40)), old=block * first, new=block * blocks, dim=dim,
                    block=block, factor=rng.choice([2, 3, 4, 8]))
    block = rng.choice([64, 64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 8])
    batch = rng.choice([1, 2, 5, 8, 24])
    drafts = rng.choice([1, 1, 2, 7, 16, 33, 64])
    bits = rng.choice([8, 8, 16])
    if rng.random() < 0.5:
        tail = _spread(rng, 1, max(2, 200000 // (batch * hkv)))
        cap, seq, topk = block * ((tail + block - 1) // block + rng.randrange(0, 3)), 0, 0
    else:
        blocks = _spread(rng, 4, 256)
        topk = min(rng.choice([1, 5, 16, 64]), blocks)
        seq, tail = block * blocks, rng.randrange(0, 3 * block)
        cap = seq + 3 * block
    return dict(kind="tree", batch=batch, hq=hkv * group, hkv=hkv, drafts=drafts, cap=cap, seq=seq, tail=tail,
                dim=dim, block=block, topk=topk, per_qhead=topk > 0 and rng.random() < 0.25, bits=bits,
                branchy=drafts > 1 and rng.random() < 0.8)


# ------------------------------------------------------------------------------------ the inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _int(g, lo, hi, shape):
    return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=torch.int32)


def _levels(n, factor):
    sizes = [n]
    while sizes[-1] > factor:
        sizes.append(-(-sizes[-1] // factor))
    return sizes


def _fill(g, case, with_v=True):
    """Cache buffers of `case` with rows in all of the capacity: 64 clusters of keys per plane, one
    per run of 64 keys, and values of like size; as 8-bit values and exponents, or bf16."""
    b, h, cap, d = case["batch"], case["hkv"], case["cap"], case["dim"]
    fp8 = case["bits"] == 8 if "bits" in case else True
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    out = {}
    for name in ("k", "v") if with_v else ("k",):
        buf = torch.empty((b, h, cap, d), dtype=dt, device=DEV)
        exps = torch.empty((b, h, cap), dtype=torch.uint8, device=DEV) if fp8 else None
        for i in range(b):
            x = _randn(g, h, cap, d)
            if name == "k":
                cent = _randn(g, h, 64, d)
                cid = torch.randint(0, 64, (h, -(-cap // 64)), generator=g, device=DEV)
                run = cid.repeat_interleave(64, dim=1)[:, :cap]
                x = x.mul_(0.3).add_(cent.gather(1, run[..., None].expand(-1, -1, d)))
            x = x.to(torch.bfloat16)
            if fp8:
                q, e = _quantised(x)
                buf[i] = q
                exps[i] = e
            else:
                buf[i] = x
        out[name], out[name + "_exp"] = buf, exps
    return out


def prepare(case, seed):
    g = _gen(seed)
    kind = case["kind"]
    s = {"case": case, "kept": {}}
    if kind == "rope":
        b, t, hq, hkv, d = (case[x] for x in ("batch", "tokens", "hq", "hkv", "dim"))
        packed = torch.empty((b, t, (hq + 2 * hkv) * d), dtype=torch.bfloat16, device=DEV)
        packed.normal_(generator=g)
        packed = packed.view(b, t, hq + 2 * hkv, d)
        s["xq"], s["xk"] = packed[:, :, :hq], packed[:, :, hq:hq + hkv]
        s["wq"] = (1 + 0.2 * _randn(g, d)) if case["weights"] else None
        s["wk"] = (1 + 0.2 * _randn(g, d)) if case["weights"] else None
        i = torch.arange(case["rot"] // 2, device=DEV, dtype=torch.float64)
        s["inv_freq"] = (10000.0 ** (-2.0 * i / case["rot"])).float()
        first = _int(g, 0, max(1, case["far"]), (b, 1))
        s["pos"] = (first + torch.arange(t, device=DEV, dtype=torch.int32)).to(torch.int32).contiguous()
        if case["backward"]:
            s["dq"] = torch.empty((b, hq, t, d), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
            s["dk"] = torch.empty((b, hkv, t, d), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
        return s
    if kind == "pyramid":
        s.update(_fill(g, case, with_v=False))
        sizes = _levels(case["cap"] // case["block"], case["factor"])
        s["pyramid"] = torch.zeros((case["batch"], case["hkv"], sum(sizes), case["dim"]), device=DEV)
        _pyramid_plain(s, 0, case["old"])       # the pyramid of the cache before its new blocks
        return s
    s.update(_fill(g, case))
    b, hkv, d, cap = case["batch"], case["hkv"], case["dim"], case["cap"]
    if kind in ("write", "read"):
        t = case["tokens"]
        if case["ragged"]:
            s["start"] = _int(g, 0, cap - t + 1, (b,))
            s["count"] = _int(g, (t + 1) // 2, t + 1, (b,))
        else:
            s["start"], s["count"] = None, None
        if kind == "write":
            s["new_k"] = _randn(g, b, hkv, t, d).to(torch.bfloat16)
            packed = _randn(g, b, t, 2 * hkv, d).to(torch.bfloat16)   # V stays in the projection's layout
            s["new_v"] = packed[:, :, hkv:].transpose(1, 2)
        else:
            s["out_k"] = torch.zeros((b, hkv, t, d), dtype=torch.bfloat16, device=DEV)
            s["out_v"] = torch.zeros((b, hkv, t, d), dtype=torch.bfloat16, device=DEV)
        return s
    hq, t = case["hq"], case["drafts"]
    s["q"] = (1.5 * _randn(g, b, hq, t, d)).to(torch.bfloat16)
    s["dk"] = _randn(g, b, hkv, t, d).to(torch.bfloat16)
    s["dv"] = _randn(g, b, hkv, t, d).to(torch.bfloat16)
    # each drafted token's parent is an earlier one (branchy) or the one before it; ancestors and itself
    parent = torch.arange(t) - 1
    if case["branchy"]:
        r = torch.rand(t, generator=torch.Generator().manual_seed(int(seed)))
        parent = torch.minimum(parent, (r * torch.arange(t)).long())
    rows = []
    for i in range(t):
        m = 1 << i
        if i > 0:
            m |= rows[int(max(0, parent[i]))]
        rows.append(m)
    s["mask"] = torch.tensor([m - (1 << 64) if m >> 63 else m for m in rows], dtype=torch.int64, device=DEV) \
        .expand(b, t).contiguous()
    lo = case["seq"] if case["topk"] else case["tail"] // 3
    s["len"] = _int(g, lo, case["seq"] + case["tail"] + 1, (b,))
    s["idx"] = None
    if case["topk"]:
        hsel = hq if case["per_qhead"] else hkv
        n = case["seq"] // case["block"]
        pick = torch.rand((b, hsel, n), generator=g, device=DEV).topk(case["topk"], dim=-1).indices
        s["idx"] = pick.sort(dim=-1).values.to(torch.int32)[:, :, None].contiguous()
    return s


# ------------------------------------------------------------------------------------ plain forms

def _rotated(y, cos, sin, rot, interleaved, back):
    """Rotates the first `rot` dims of y [..., D]; pairs (2i, 2i+1) or (i, i + rot/2)."""
    if rot == 0:
        return y
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    sn = -sin if back else sin
    u, v = a * cos - b * sn, a * sn + b * cos
    turned = torch.stack((u, v), dim=-1).flatten(-2) if interleaved else torch.cat((u, v), dim=-1)
    return torch.cat((turned, y[..., rot:]), dim=-1)


def _angles(s):
    a = s["pos"].double()[..., None] * s["inv_freq"].double()     # [B, T, rot / 2]
    return a.cos().float()[:, :, None], a.sin().float()[:, :, None]


def _norm_rope_plain(x, w, s):
    c = s["case"]
    cos, sin = _angles(s)
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    y = y * w if w is not None else y
    y = _rotated(y, cos, sin, c["rot"], c["interleaved"], False)
    return y.transpose(1, 2).to(torch.bfloat16).contiguous()


def _norm_rope_grad_plain(x, w, dy, s):
    c = s["case"]
    cos, sin = _angles(s)
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    xh = x * r
    dy = _rotated(dy.transpose(1, 2).float(), cos, sin, c["rot"], c["interleaved"], True)
    dw = (dy * xh).sum(dim=2).sum(dim=1).sum(dim=0) if w is not None else None
    dh = dy * w if w is not None else dy
    dx = r * (dh - xh * (dh * xh).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), dw


def _pow2(exps):
    """2^(e - 127) of exponent bytes 1..254, from its bits (exact)."""
    return (exps.to(torch.int32) << 23).view(torch.float32)


def _quantised(x):
    """bf16 rows [..., D] -> e4m3 values and the exponent byte e of each row: x ~ value * 2^(e - 127),
    2^(e - 127) the smallest power of two with |x| / 2^(e - 127) <= 448 (e >= 1)."""
    x = x.float()
    top = x.abs().amax(-1)
    m, k = torch.frexp(top)                                    # top = m 2^k, m in [0.5, 1)
    e = k - 9 + (m > 0.875).int()                              # 448 = 0.875 * 2^9
    e = torch.where(top > 0, e, torch.full_like(e, -126)).clamp(min=-126)
    q = (x * _pow2(127 - e)[..., None]).to(torch.float8_e4m3fn)
    return q, (e + 127).to(torch.uint8)


def _values(q, exps):
    x = q.float()
    return x if exps is None else x * _pow2(exps)[..., None]


def _slots(s):
    """Cache positions of the call's rows and which of them count, [B, T] each."""
    c = s["case"]
    t = torch.arange(c["tokens"], device=DEV)
    if s["start"] is None:
        return t.expand(c["batch"], -1), torch.ones((c["batch"], c["tokens"]), dtype=torch.bool, device=DEV)
    return s["start"].long()[:, None] + t, t < s["count"][:, None]


def _put(buf, pos, keep, new):
    """buf[b, :, pos[b, t]] = new[b, :, t] where keep[b, t] (the old row is written back elsewhere)."""
    at = torch.arange(buf.shape[0], device=DEV)[:, None]
    rows = buf.transpose(1, 2)
    old = rows[at, pos]
    rows[at, pos] = torch.where(keep.view(*keep.shape, *[1] * (old.dim() - 2)), new.transpose(1, 2), old)


def _write_plain(s):
    pos, keep = _slots(s)
    out = [s["k"], s["v"]]
    if s["k_exp"] is None:
        _put(s["k"], pos, keep, s["new_k"])
        _put(s["v"], pos, keep, s["new_v"])
        return out
    qk, ek = _quantised(s["new_k"])
    qv, ev = _quantised(s["new_v"])
    _put(s["k"].view(torch.uint8), pos, keep, qk.view(torch.uint8))
    _put(s["v"].view(torch.uint8), pos, keep, qv.view(torch.uint8))
    _put(s["k_exp"], pos, keep, ek)
    _put(s["v_exp"], pos, keep, ev)
    return out + [s["k_exp"], s["v_exp"]]


def _rows_plain(buf, exps, pos, keep, out):
    at = torch.arange(buf.shape[0], device=DEV)[:, None]
    if exps is None:
        x = buf.transpose(1, 2)[at, pos]
    else:
        q = buf.view(torch.uint8).transpose(1, 2)[at, pos].view(torch.float8_e4m3fn)
        x = _values(q, exps.transpose(1, 2)[at, pos]).to(torch.bfloat16)
    out.copy_(torch.where(keep[:, None, :, None], x.transpose(1, 2), out))
    return out


def _pyramid_plain(s, old, new):
    """Level-0 means of the blocks [old, new) and, level after level, the nodes over them, each the
    mean of all keys that it covers so far."""
    c = s["case"]
    b, h, d, blk, f = c["batch"], c["hkv"], c["dim"], c["block"], c["factor"]
    if new == old:
        return s["pyramid"]
    lo, hi, off, width = old // blk, new // blk, 0, 1
    k = _values(s["k"][:, :, old:new].contiguous(), s["k_exp"][:, :, old:new])
    s["pyramid"][:, :, lo:hi] = k.view(b, h, hi - lo, blk, d).mean(3)
    valid = new // blk
    for n in _levels(c["cap"] // blk, f)[:-1]:
        w = width * f
        c_lo, c_hi = (old // blk) // w, (valid - 1) // w + 1
        child = torch.arange(c_lo * f, min(c_hi * f, n), device=DEV)
        weight = (valid - child * width).clamp(0, width).float()
        pad = (c_hi - c_lo) * f - child.numel()
        x = s["pyramid"][:, :, off:off + n][:, :, c_lo * f:c_lo * f + child.numel()] * weight[:, None]
        x = torch.nn.functional.pad(x, (0, 0, 0, pad)).view(b, h, c_hi - c_lo, f, d).sum(3)
        total = torch.nn.functional.pad(weight, (0, pad)).view(-1, f).sum(-1)
        s["pyramid"][:, :, off + n + c_lo:off + n + c_hi] = x / total[:, None]
        off, width = off + n, w
    return s["pyramid"]


def _selected(s, name):
    """Keys (or values) of every selection row: the listed blocks, then the tail, and their positions
    (-1 where a list entry is empty). [B, Hsel, n, D] in fp32 and [B, Hsel, n]."""
    c = s["case"]
    buf, exps = s[name], s[name + "_exp"]
    b, hkv, cap, d = buf.shape
    hsel = c["hq"] if c["per_qhead"] else hkv
    head = torch.arange(hsel, device=DEV) // (hsel // hkv)
    tail = slice(c["seq"], c["seq"] + c["tail"])
    x = _values(buf[:, :, tail], None if exps is None else exps[:, :, tail])
    pos = torch.arange(c["seq"], c["seq"] + c["tail"], device=DEV).expand(b, hsel, -1)
    x = x[:, head] if c["per_qhead"] else x
    if not c["topk"]:
        return x, pos
    blk = c["block"]
    idx = s["idx"][:, :, 0].long()
    at = (torch.arange(b, device=DEV)[:, None, None], head[None, :, None], idx.clamp(min=0))
    raw = buf if exps is None else buf.view(torch.uint8)
    got = raw.view(b, hkv, cap // blk, blk, d)[at].reshape(b, hsel, -1, d)
    if exps is not None:
        e = exps.view(b, hkv, cap // blk, blk)[at].reshape(b, hsel, -1)
        got = _values(got.view(torch.float8_e4m3fn), e)
    p = idx[..., None] * blk + torch.arange(blk, device=DEV)
    p = torch.where(idx[..., None] >= 0, p, -1).reshape(b, hsel, -1)
    return torch.cat((got.float(), x), dim=2), torch.cat((p, pos), dim=2)


def _tree_plain(s):
    c = s["case"]
    b, hq, t, d = s["q"].shape
    hsel = hq if c["per_qhead"] else c["hkv"]
    gh = hq // hsel
    k, pos = _selected(s, "k")
    v, _ = _selected(s, "v")
    head = torch.arange(hsel, device=DEV) // (hsel // c["hkv"])
    k = torch.cat((k, s["dk"][:, head].float()), dim=2)
    v = torch.cat((v, s["dv"][:, head].float()), dim=2)
    seen = (pos >= 0) & (pos < s["len"][:, None, None])
    bits = (s["mask"][:, :, None] >> torch.arange(t, device=DEV)) & 1
    seen = torch.cat((seen[:, :, None].expand(-1, -1, t, -1), (bits == 1)[:, None].expand(-1, hsel, -1, -1)), dim=-1)
    q = s["q"].float().view(b, hsel, gh * t, d)
    x = (q @ k.transpose(-1, -2) / math.sqrt(d)).view(b, hsel, gh, t, -1)
    x = x.masked_fill_(~seen[:, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1)
    o = (x.view(b, hsel, gh * t, -1) @ v).view(b, hsel, gh, t, d)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    lse = top[..., 0] + total.log()
    return o.reshape(b, hq, t, d).to(torch.bfloat16), lse.reshape(b, hq, t)


# ------------------------------------------------------------------------------------ one pass

def _keep(s, name, make):
    """What a serving program makes once and keeps: shapes, the cache's handle, workspaces."""
    if name not in s["kept"]:
        s["kept"][name] = make()
    return s["kept"][name]


def _rope_shape(pisa, c):
    return pisa.NormRopeShape(batch=c["batch"], tokens=c["tokens"], heads_q=c["hq"], heads_kv=c["hkv"],
                              head_dim=c["dim"], rotary_dim=c["rot"], interleaved=int(c["interleaved"]), eps=1e-6)


def _cache(pisa, s):
    c = s["case"]
    fmt = pisa.CACHE_BF16 if s["k_exp"] is None else pisa.CACHE_E4M3
    shape = pisa.CacheShape(batch=c["batch"], heads_kv=c["hkv"], capacity=c["cap"], head_dim=c["dim"], format=fmt)
    return pisa.Cache(shape, s["k"], s.get("v"), s["k_exp"], s.get("v_exp"))


def _run_own(s):
    import block_sparse_long_pisa_b200 as pisa
    c = s["case"]
    if c["kind"] == "rope":
        shape = _keep(s, "shape", lambda: _rope_shape(pisa, c))
        if not c["backward"]:
            return pisa.qk_norm_rope(shape, s["xq"], s["xk"], s["pos"], s["inv_freq"], s["wq"], s["wk"])
        ws = _keep(s, "ws", lambda: pisa.new_norm_rope_workspace(shape, DEV))
        return pisa.qk_norm_rope_backward(shape, s["xq"], s["xk"], s["pos"], s["inv_freq"], s["dq"], s["dk"],
                                          s["wq"], s["wk"], ws=ws)
    cache = _keep(s, "cache", lambda: _cache(pisa, s))
    if c["kind"] == "pyramid":
        shape = _keep(s, "shape", lambda: pisa.Shape(c["batch"], c["hkv"], c["hkv"], 1, c["new"], c["dim"],
                                                     c["block"], c["factor"], 1, kv_capacity=c["cap"]))
        return pisa.cache_append_pyramid(shape, cache, s["pyramid"], c["old"])
    if c["kind"] == "tree":
        shape = _keep(s, "shape", lambda: pisa.TreeShape(
            batch=c["batch"], heads_q=c["hq"], heads_kv=c["hkv"], drafts=c["drafts"], capacity=c["cap"],
            head_dim=c["dim"], format=cache.shape.format, block=c["block"], seq_kv=c["seq"], topk=c["topk"],
            select_per_qhead=int(c["per_qhead"])))
        ws = _keep(s, "ws", lambda: pisa.new_tree_workspace(shape, DEV))
        return pisa.tree_attention(shape, cache, s["q"], s["dk"], s["dv"], s["mask"], s["len"], ws, idx=s["idx"])
    ws = _keep(s, "ws", lambda: pisa.new_cache_workspace(DEV))
    if c["kind"] == "write":
        pisa.cache_write(cache, s["new_k"], s["new_v"], ws, start=s["start"], count=s["count"])
        return [x for x in (s["k"], s["v"], s["k_exp"], s["v_exp"]) if x is not None]
    return pisa.cache_read(cache, c["tokens"], ws, start=s["start"], count=s["count"], K=s["out_k"], V=s["out_v"])


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["kind"] == "rope":
        if not c["backward"]:
            return _norm_rope_plain(state["xq"], state["wq"], state), _norm_rope_plain(state["xk"], state["wk"], state)
        dxq, dwq = _norm_rope_grad_plain(state["xq"], state["wq"], state["dq"], state)
        dxk, dwk = _norm_rope_grad_plain(state["xk"], state["wk"], state["dk"], state)
        return dxq, dxk, dwq, dwk
    if c["kind"] == "write":
        return _write_plain(state)
    if c["kind"] == "read":
        pos, keep = _slots(state)
        return (_rows_plain(state["k"], state["k_exp"], pos, keep, state["out_k"]),
                _rows_plain(state["v"], state["v_exp"], pos, keep, state["out_v"]))
    if c["kind"] == "pyramid":
        return _pyramid_plain(state, c["old"], c["new"])
    return _tree_plain(state)


def work(case):
    c = case
    if c["kind"] == "rope":
        x = c["batch"] * c["tokens"] * (c["hq"] + c["hkv"]) * c["dim"]
        return {"bytes": x * 2 * (3 if c["backward"] else 2) + 4 * c["batch"] * c["tokens"],
                "flops": x * (20 if c["backward"] else 9)}
    if c["kind"] in ("write", "read"):
        rows = 2 * c["batch"] * c["hkv"] * c["tokens"] * (0.75 if c["ragged"] and c["tokens"] > 1 else 1)
        one = c["dim"] + 1 if c["bits"] == 8 else 2 * c["dim"]
        return {"bytes": rows * (2 * c["dim"] + one), "flops": rows * c["dim"] * 2}
    if c["kind"] == "pyramid":
        planes, new = c["batch"] * c["hkv"], c["new"] - c["old"]
        return {"bytes": planes * (new * (c["dim"] + 1) + new // c["block"] * c["dim"] * 4),
                "flops": planes * new * c["dim"] * 2}
    hsel = c["hq"] if c["per_qhead"] else c["hkv"]
    cached = c["topk"] * c["block"] + c["tail"] / 2 if c["topk"] else c["tail"] * 2 / 3
    one = c["dim"] + 1 if c["bits"] == 8 else 2 * c["dim"]
    rows = c["batch"] * c["hq"] * c["drafts"]
    kv = c["batch"] * (hsel * c["topk"] * c["block"] + c["hkv"] * (cached - c["topk"] * c["block"]))
    return {"bytes": 2 * kv * one + 4 * c["batch"] * c["hkv"] * c["drafts"] * c["dim"] + rows * (4 * c["dim"] + 4),
            "flops": 4 * c["dim"] * rows * (cached + c["drafts"] / 2)}


# ------------------------------------------------------------------------------------ 64-bit definitions

def _exact_rope(s):
    c = s["case"]
    d, rot = c["dim"], c["rot"]
    freq = s["inv_freq"].double()
    # each output dim as a combination of two normalised dims: y[i] = a[i] u[i] + b[i] u[mate[i]]
    dim = torch.arange(d, device=DEV)
    if c["interleaved"]:
        pair, second, mate = dim // 2, dim % 2 == 1, dim ^ 1
    else:
        pair, second = dim % max(1, rot // 2), dim >= rot // 2
        mate = torch.where(second, dim - rot // 2, dim + rot // 2)
    turned = dim < rot
    pair, mate = torch.where(turned, pair, 0), torch.where(turned, mate, dim)
    angle = s["pos"].double()[..., None] * freq[pair] if rot else torch.zeros((*s["pos"].shape, d), device=DEV).double()
    ca = torch.where(turned, angle.cos(), 1.0)[:, :, None]
    sb = torch.where(turned, torch.where(second, angle.sin(), -angle.sin()), 0.0)[:, :, None]

    def one(x, w, dy):
        outs = []
        for lo in range(0, x.shape[1], 8192):
            sl = slice(lo, lo + 8192)
            xx = x[:, sl].double()
            scale = (xx.pow(2).sum(-1, keepdim=True) / d + 1e-6).pow(-0.5)
            wd = torch.ones(d, device=DEV).double() if w is None else w.double()
            a, b = ca[:, sl], sb[:, sl]
            if dy is None:
                u = xx * scale * wd
                outs.append((a * u + b * u[..., mate]).transpose(1, 2))
                continue
            g = dy[:, :, sl].transpose(1, 2).double()
            du = a * g + (b * g)[..., mate]
            n = xx * scale
            dn = du * wd
            dx = scale * dn - xx * scale.pow(3) * (dn * xx).sum(-1, keepdim=True) / d
            outs.append((dx, torch.einsum("bthd,bthd->d", du, n)))
        if dy is None:
            return torch.cat(outs, dim=2)
        return torch.cat([o[0] for o in outs], dim=1), (sum(o[1] for o in outs) if w is not None else None)

    if not c["backward"]:
        return one(s["xq"], s["wq"], None), one(s["xk"], s["wk"], None)
    (dxq, dwq), (dxk, dwk) = one(s["xq"], s["wq"], s["dq"]), one(s["xk"], s["wk"], s["dk"])
    return dxq, dxk, dwq, dwk


def _two_to(e):
    """2^e in 64 bits for whole e, from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_quantise(x):
    x = x.double()
    top = x.abs().max(dim=-1, keepdim=True).values
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 448))
    e = e + (top > 448 * _two_to(e)).double()              # where log2 was rounded over a border
    e = e - (top <= 448 * _two_to(e - 1)).double()
    e = torch.where(top > 0, e, -126.0).clamp(min=-126.0)
    y = x / _two_to(e)
    step = _two_to(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, e[..., 0] + 127


def _exact_values(q, exps):
    return q.double() if exps is None else q.double() * _two_to(exps.double() - 127)[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["kind"] == "rope":
        return _exact_rope(s)
    if c["kind"] in ("write", "read"):
        outs = []
        for name in ("k", "v"):
            buf, exps = s[name], s[name + "_exp"]
            if c["kind"] == "read":
                out = s["out_" + name].double()
            else:
                out, oe = buf.double(), None if exps is None else exps.clone()
                new = s["new_" + name]
                q, e = (new.double(), None) if exps is None else _exact_quantise(new)
            for b in range(c["batch"]):
                a = 0 if s["start"] is None else int(s["start"][b])
                n = c["tokens"] if s["count"] is None else int(s["count"][b])
                if c["kind"] == "read":
                    out[b, :, :n] = _exact_values(buf[b, :, a:a + n], None if exps is None else exps[b, :, a:a + n])
                else:
                    out[b, :, a:a + n] = q[b, :, :n]
                    if e is not None:
                        oe[b, :, a:a + n] = e[b, :, :n].to(torch.uint8)
            outs.append((out, oe if c["kind"] == "write" else None))
        return [o for o, _ in outs] + [e for _, e in outs if e is not None]
    if c["kind"] == "pyramid":
        n, total, planes = c["new"] // c["block"], c["cap"] // c["block"], []
        keys = _exact_values(s["k"][:, :, :c["new"]].contiguous(), s["k_exp"][:, :, :c["new"]])
        sums = torch.cumsum(keys.view(*keys.shape[:2], n, c["block"], c["dim"]).sum(3), dim=2)
        sums = torch.cat((torch.zeros_like(sums[:, :, :1]), sums), dim=2)      # keys before block i
        for level, size in enumerate(_levels(total, c["factor"])):
            lo = (torch.arange(size, device=DEV) * c["factor"] ** level).clamp(max=n)
            hi = ((torch.arange(size, device=DEV) + 1) * c["factor"] ** level).clamp(max=n)
            keys_in = ((hi - lo) * c["block"]).clamp(min=1).double()
            planes.append((sums[:, :, hi] - sums[:, :, lo]) / keys_in[:, None])
        return torch.cat(planes, dim=2)
    b, hq, t, d = s["q"].shape
    o = torch.zeros((b, hq, t, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((b, hq, t), dtype=torch.float64, device=DEV)
    group = hq // c["hkv"]
    own_bits = ((s["mask"][:, :, None] >> torch.arange(t, device=DEV)) & 1).bool()
    for i in range(b):
        n = int(s["len"][i])
        for h in range(hq):
            kv = h // group
            where = torch.arange(min(c["seq"], n) if c["topk"] else 0, n, device=DEV)
            if c["topk"]:
                blocks = s["idx"][i, h if c["per_qhead"] else kv, 0].long()
                at = (blocks[blocks >= 0, None] * c["block"] + torch.arange(c["block"], device=DEV)).flatten()
                where = torch.cat((at[at < n], where))
            ek = None if s["k_exp"] is None else s["k_exp"][i, kv, where]
            ev = None if s["v_exp"] is None else s["v_exp"][i, kv, where]
            kk = torch.cat((_exact_values(_take(s["k"][i, kv], where), ek), s["dk"][i, kv].double()))
            vv = torch.cat((_exact_values(_take(s["v"][i, kv], where), ev), s["dv"][i, kv].double()))
            x = s["q"][i, h].double() @ kk.T * (d ** -0.5)
            x[:, where.numel():].masked_fill_(~own_bits[i], -math.inf)
            lse[i, h] = torch.logsumexp(x, dim=-1)
            o[i, h] = torch.softmax(x, dim=-1) @ vv
    return o, lse


def _take(rows, where):
    if rows.dtype == torch.float8_e4m3fn:
        return rows.view(torch.uint8)[where].view(torch.float8_e4m3fn)
    return rows[where]
