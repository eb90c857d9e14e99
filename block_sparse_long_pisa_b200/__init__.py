"""Python binding of libpisa.so (PISA pyramid block-sparse attention for B200).

Argument marshalling only: every step of the method runs in the CUDA kernels
behind the C ABI of include/pisa.h. PyTorch supplies device memory and the
current stream. There is no CPU fallback: importing this package fails if the
compiled library is missing, and every call raises PisaError on a non-OK
status.
"""
from __future__ import annotations

import ctypes
import dataclasses
import math
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpisa.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libpisa.so is not built ({LIB_PATH}); run __graft_entry__.build() first")
_lib = ctypes.CDLL(LIB_PATH)

MAX_LEVELS = 24
MAX_CANDIDATES = 4096

STATUS = {0: "PISA_OK", 1: "PISA_ERR_INVALID_ARG", 2: "PISA_ERR_UNSUPPORTED", 3: "PISA_ERR_WORKSPACE",
          4: "PISA_ERR_CUDA", 5: "PISA_ERR_TIMEOUT", 6: "PISA_ERR_BAD_INDEX"}
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT, ERR_BAD_INDEX = range(7)


class PisaShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "heads_q", "heads_kv", "seq_q", "seq_kv", "head_dim",
                                               "block", "factor", "topk", "causal", "select_per_qhead")] + \
               [("scale", ctypes.c_float), ("forced_blocks", ctypes.c_int32), ("kv_capacity", ctypes.c_int32)]

FORCE_SINK, FORCE_LOCAL = 1, 2   # pisa_shape.forced_blocks bits


_i64x3 = ctypes.c_int64 * 3


class PisaNormRopeShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "tokens", "heads_q", "heads_kv", "head_dim", "rotary_dim",
                                               "interleaved")] + \
               [("eps", ctypes.c_float)] + [(n, _i64x3) for n in ("xq_stride", "xk_stride", "dxq_stride", "dxk_stride")]


class PisaCacheShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "heads_kv", "capacity", "head_dim", "format")]


class PisaTreeShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "heads_q", "heads_kv", "drafts", "capacity", "head_dim", "format",
                                               "block", "seq_kv", "topk", "select_per_qhead")] + \
               [("scale", ctypes.c_float)]

CACHE_BF16, CACHE_E4M3 = 0, 1   # pisa_cache_shape.format


class PisaError(RuntimeError):
    def __init__(self, status: int, where: str, detail: int | None = None):
        self.status = status
        self.detail = detail
        msg = f"{where}: {STATUS.get(status, status)} ({_lib.pisa_status_string(status).decode()})"
        if detail is not None:
            msg += f" detail=0x{detail:x}"
        super().__init__(msg)


_vp, _i32p, _f32p, _szp = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32), ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)
_SP = ctypes.POINTER(PisaShape)
_NP, _CP, _TP = ctypes.POINTER(PisaNormRopeShape), ctypes.POINTER(PisaCacheShape), ctypes.POINTER(PisaTreeShape)
_sig = {
    "pisa_num_levels": (ctypes.c_int32, [_SP]),
    "pisa_level_layout": (ctypes.c_int, [_SP, _i32p, _i32p]),
    "pisa_pyramid_size": (ctypes.c_int, [_SP, _szp]),
    "pisa_workspace_size": (ctypes.c_int, [_SP, _szp]),
    "pisa_build_pyramid": (ctypes.c_int, [_SP, _vp, _vp, _vp]),
    "pisa_append_pyramid": (ctypes.c_int, [_SP, _vp, _vp, ctypes.c_int32, _vp]),
    "pisa_backward_workspace_size": (ctypes.c_int, [_SP, _szp]),
    "pisa_sparse_attention_backward": (ctypes.c_int, [_SP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                      ctypes.c_size_t, _vp]),
    "pisa_select_blocks": (ctypes.c_int, [_SP, _vp, _vp, _i32p, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "pisa_sparse_attention": (ctypes.c_int, [_SP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "pisa_forward": (ctypes.c_int, [_SP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "pisa_check_status": (ctypes.c_int, [_vp, ctypes.POINTER(ctypes.c_uint32), _vp]),
    "pisa_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "pisa_last_launch_count": (ctypes.c_int32, []),
    "pisa_decode_attention_noalloc": (ctypes.c_int, [_SP, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "pisa_decode_noalloc_check_status": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint32), _vp]),
    "pisa_qk_norm_rope": (ctypes.c_int, [_NP] + [_vp] * 9),
    "pisa_norm_rope_workspace_size": (ctypes.c_int, [_NP, _szp]),
    "pisa_qk_norm_rope_backward": (ctypes.c_int, [_NP] + [_vp] * 13 + [ctypes.c_size_t, _vp]),
    "pisa_cache_write": (ctypes.c_int, [_CP, ctypes.c_int32, _vp, _vp, _i64x3, _i64x3] + [_vp] * 8),
    "pisa_cache_read": (ctypes.c_int, [_CP, ctypes.c_int32] + [_vp] * 10),
    "pisa_cache_append_pyramid": (ctypes.c_int, [_SP, _vp, _vp, _vp, ctypes.c_int32, _vp]),
    "pisa_tree_workspace_size": (ctypes.c_int, [_TP, _szp]),
    "pisa_tree_attention": (ctypes.c_int, [_TP] + [_vp] * 13 + [ctypes.c_size_t, _vp]),
    "pisa_selftest_wait_timeout": (ctypes.c_int, [_vp, ctypes.c_uint32, _vp]),
}
for _name, (_res, _args) in _sig.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_sig)


@dataclasses.dataclass(frozen=True)
class Shape:
    """Problem description (mirrors pisa_shape)."""
    batch: int
    heads_q: int
    heads_kv: int
    seq_q: int
    seq_kv: int
    head_dim: int
    block: int
    factor: int
    topk: int
    causal: int = 0
    select_per_qhead: int = 0
    scale: float = 0.0
    forced_blocks: int = 0   # FORCE_SINK | FORCE_LOCAL
    kv_capacity: int = 0     # decode over a growing cache: K/V rows per plane (0 = seq_kv)

    def c(self) -> PisaShape:
        return PisaShape(self.batch, self.heads_q, self.heads_kv, self.seq_q, self.seq_kv, self.head_dim,
                         self.block, self.factor, self.topk, int(self.causal), int(self.select_per_qhead),
                         float(self.scale), int(self.forced_blocks), int(self.kv_capacity))

    @property
    def decode(self) -> bool:
        return self.seq_q == 1

    @property
    def n_blocks(self) -> int:
        return self.seq_kv // self.block

    @property
    def kv_rows(self) -> int:
        """Rows of one K/V plane: the capacity of a growing cache, else seq_kv."""
        return self.kv_capacity or self.seq_kv

    @property
    def n_nodes(self) -> int:
        """Rows of one pyramid plane: level sizes n_0 = kv_rows / block, ceil(n / factor) while n > factor."""
        n = total = self.kv_rows // self.block
        while n > self.factor >= 2:
            n = -(-n // self.factor)
            total += n
        return total

    @property
    def hsel(self) -> int:
        return self.heads_q if self.select_per_qhead else self.heads_kv

    @property
    def n_qblocks(self) -> int:
        return 1 if self.decode else self.seq_q // self.block

    @classmethod
    def of(cls, w, **kw) -> "Shape":
        """Shape of a workload description (any object with the same field names)."""
        f = {k: getattr(w, k) for k in ("batch", "heads_q", "heads_kv", "seq_q", "seq_kv", "head_dim", "block",
                                        "factor", "topk", "causal")}
        f.update(kw)
        return cls(**f)


def _check(status: int, where: str) -> None:
    if status != OK:
        raise PisaError(status, where)


def num_levels(shape: Shape) -> int:
    return int(_lib.pisa_num_levels(ctypes.byref(shape.c())))


def level_layout(shape: Shape) -> tuple[list[int], list[int]]:
    sizes = (ctypes.c_int32 * MAX_LEVELS)()
    offs = (ctypes.c_int32 * MAX_LEVELS)()
    _check(_lib.pisa_level_layout(ctypes.byref(shape.c()), sizes, offs), "pisa_level_layout")
    n = num_levels(shape)
    return list(sizes[:n]), list(offs[:n])


def pyramid_size(shape: Shape) -> int:
    n = ctypes.c_size_t()
    _check(_lib.pisa_pyramid_size(ctypes.byref(shape.c()), ctypes.byref(n)), "pisa_pyramid_size")
    return n.value


def workspace_size(shape: Shape) -> int:
    n = ctypes.c_size_t()
    _check(_lib.pisa_workspace_size(ctypes.byref(shape.c()), ctypes.byref(n)), "pisa_workspace_size")
    return n.value


def last_launch_count() -> int:
    return int(_lib.pisa_last_launch_count())


# ----------------------------------------------------------------------------- torch-facing calls

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _made(stream, make):
    """make(), a tensor of a call that runs on `stream` (None: the current one): allocated and filled there, so that
    neither the fill nor a later owner of freed memory can meet the call's kernels. It is returned to work on the
    caller's current stream, which its memory is kept for too."""
    if stream is None:
        return make()
    torch = _torch()
    mine = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        t = make()
    if mine != stream:
        t.record_stream(mine)
    return t


def _need(t, dtype, shape, name):
    torch = _torch()
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def new_workspace(shape: Shape, device) -> "object":
    """Zeroed workspace (the status word must start at zero)."""
    torch = _torch()
    return torch.zeros(workspace_size(shape), dtype=torch.uint8, device=device)


def build_pyramid(shape: Shape, K, pyramid=None, stream=None):
    torch = _torch()
    D = shape.head_dim
    _need(K, torch.bfloat16, (shape.batch, shape.heads_kv, shape.kv_rows, D), "K")
    sizes, _ = level_layout(shape)
    if pyramid is None:
        pyramid = _made(stream, lambda: torch.empty((shape.batch, shape.heads_kv, sum(sizes), D), dtype=torch.float32,
                                                    device=K.device))
    _check(_lib.pisa_build_pyramid(ctypes.byref(shape.c()), _ptr(K), _ptr(pyramid), _stream(stream)),
           "pisa_build_pyramid")
    return pyramid


def append_pyramid(shape: Shape, K, pyramid, seq_kv_old: int, stream=None):
    """Brings `pyramid` (the pyramid of the cache at length seq_kv_old) up to shape.seq_kv."""
    torch = _torch()
    _need(K, torch.bfloat16, (shape.batch, shape.heads_kv, shape.kv_rows, shape.head_dim), "K")
    _check(_lib.pisa_append_pyramid(ctypes.byref(shape.c()), _ptr(K), _ptr(pyramid), int(seq_kv_old), _stream(stream)),
           "pisa_append_pyramid")
    return pyramid


def select_blocks(shape: Shape, Q, pyramid, ws, level_budget=None, idx=None, margin=False, stream=None):
    torch = _torch()
    _need(Q, torch.bfloat16, (shape.batch, shape.heads_q, shape.seq_q, shape.head_dim), "Q")
    if idx is None:
        idx = _made(stream, lambda: torch.empty((shape.batch, shape.hsel, shape.n_qblocks, shape.topk), dtype=torch.int32,
                                                device=Q.device))
    marg = _made(stream, lambda: torch.empty((shape.batch, shape.hsel, shape.n_qblocks), dtype=torch.float32,
                                             device=Q.device)) if margin else None
    budget = None
    if level_budget is not None:
        budget = (ctypes.c_int32 * len(level_budget))(*[int(x) for x in level_budget])
    _check(_lib.pisa_select_blocks(ctypes.byref(shape.c()), _ptr(Q), _ptr(pyramid), budget, _ptr(idx), _ptr(marg),
                                   _ptr(ws), ws.numel(), _stream(stream)), "pisa_select_blocks")
    return (idx, marg) if margin else idx


def sparse_attention(shape: Shape, Q, K, V, idx, ws, O=None, lse=True, stream=None):
    torch = _torch()
    B, Hq, Nq, D = shape.batch, shape.heads_q, shape.seq_q, shape.head_dim
    _need(Q, torch.bfloat16, (B, Hq, Nq, D), "Q")
    if O is None:
        O = _made(stream, lambda: torch.empty_like(Q))
    L = _made(stream, lambda: torch.empty((B, Hq, Nq), dtype=torch.float32, device=Q.device)) if lse is True else lse
    _check(_lib.pisa_sparse_attention(ctypes.byref(shape.c()), _ptr(Q), _ptr(K), _ptr(V), _ptr(idx), _ptr(O),
                                      _ptr(L), _ptr(ws), ws.numel(), _stream(stream)), "pisa_sparse_attention")
    return O, L


def forward(shape: Shape, Q, K, V, ws, O=None, lse=True, idx=None, stream=None):
    """Pyramid, selection and attention in one call. Returns (O, lse, idx or None)."""
    torch = _torch()
    B, Hq, Nq, D = shape.batch, shape.heads_q, shape.seq_q, shape.head_dim
    _need(Q, torch.bfloat16, (B, Hq, Nq, D), "Q")
    _need(K, torch.bfloat16, (B, shape.heads_kv, shape.kv_rows, D), "K")
    _need(V, torch.bfloat16, (B, shape.heads_kv, shape.kv_rows, D), "V")
    if O is None:
        O = _made(stream, lambda: torch.empty_like(Q))
    L = _made(stream, lambda: torch.empty((B, Hq, Nq), dtype=torch.float32, device=Q.device)) if lse is True else lse
    if idx is True:
        idx = _made(stream, lambda: torch.empty((B, shape.hsel, shape.n_qblocks, shape.topk), dtype=torch.int32,
                                                device=Q.device))
    _check(_lib.pisa_forward(ctypes.byref(shape.c()), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(L), _ptr(idx),
                             _ptr(ws), ws.numel(), _stream(stream)), "pisa_forward")
    return O, L, idx


def decode_attention_noalloc(shape: Shape, Q, K, V, idx, O=None, lse=True, stream=None):
    """Decode attention with the library's built-in scratch (no workspace, no allocation inside)."""
    torch = _torch()
    B, Hq, D = shape.batch, shape.heads_q, shape.head_dim
    _need(Q, torch.bfloat16, (B, Hq, 1, D), "Q")
    if O is None:
        O = _made(stream, lambda: torch.empty_like(Q))
    L = _made(stream, lambda: torch.empty((B, Hq, 1), dtype=torch.float32, device=Q.device)) if lse is True else lse
    _check(_lib.pisa_decode_attention_noalloc(ctypes.byref(shape.c()), _ptr(Q), _ptr(K), _ptr(V), _ptr(idx),
                                              _ptr(O), _ptr(L), _stream(stream)), "pisa_decode_attention_noalloc")
    return O, L


def decode_noalloc_check_status(stream=None) -> tuple[int, int]:
    """Synchronises the stream; returns (status, detail) that the last decode_attention_noalloc
    call's kernels recorded in the library's built-in array, and clears them."""
    detail = ctypes.c_uint32()
    st = _lib.pisa_decode_noalloc_check_status(ctypes.byref(detail), _stream(stream))
    return int(st), int(detail.value)


def backward_workspace_size(shape: Shape) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.pisa_backward_workspace_size(ctypes.byref(shape.c()), ctypes.byref(n)), "pisa_backward_workspace_size")
    return n.value


def sparse_attention_backward(shape: Shape, Q, K, V, O, lse, dO, idx, ws=None, dQ=None, dK=None, dV=None,
                              stream=None):
    """dQ, dK, dV of the sparse attention step for the selection `idx` (prefill)."""
    torch = _torch()
    B, Hq, N, D = shape.batch, shape.heads_q, shape.seq_q, shape.head_dim
    for t, name in ((Q, "Q"), (O, "O"), (dO, "dO")):
        _need(t, torch.bfloat16, (B, Hq, N, D), name)
    for t, name in ((K, "K"), (V, "V")):
        _need(t, torch.bfloat16, (B, shape.heads_kv, shape.kv_rows, D), name)
    _need(lse, torch.float32, (B, Hq, N), "lse")
    _need(idx, torch.int32, (B, shape.hsel, shape.n_qblocks, shape.topk), "idx")
    if ws is None:
        ws = _made(stream, lambda: torch.zeros(backward_workspace_size(shape), dtype=torch.uint8, device=Q.device))
    dQ = _made(stream, lambda: torch.empty_like(Q)) if dQ is None else dQ
    dK = _made(stream, lambda: torch.empty_like(K)) if dK is None else dK
    dV = _made(stream, lambda: torch.empty_like(V)) if dV is None else dV
    _check(_lib.pisa_sparse_attention_backward(ctypes.byref(shape.c()), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(lse),
                                               _ptr(dO), _ptr(idx), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(ws), ws.numel(),
                                               _stream(stream)), "pisa_sparse_attention_backward")
    return dQ, dK, dV


def check_status(ws, stream=None) -> tuple[int, int]:
    """Synchronises the stream; returns (status, detail) recorded by kernels and clears them."""
    detail = ctypes.c_uint32()
    st = _lib.pisa_check_status(_ptr(ws), ctypes.byref(detail), _stream(stream))
    return int(st), int(detail.value)


def selftest_wait_timeout(ws, limit_us: int, stream=None) -> None:
    """Enqueues the bounded-wait self-test: a wait that never completes gives up after limit_us
    and records PISA_ERR_TIMEOUT in the workspace status word (read it with check_status)."""
    _check(_lib.pisa_selftest_wait_timeout(_ptr(ws), int(limit_us), _stream(stream)), "pisa_selftest_wait_timeout")


def raise_on_device_error(ws, where="device", stream=None) -> None:
    st, detail = check_status(ws, stream)
    if st != OK:
        raise PisaError(st, where, detail)


class Session:
    """Preallocated device buffers for repeated forwards of one shape.

    `forward` accepts host (CPU, ideally pinned) or device tensors. With host
    inputs the (batch, KV head) planes, which the method treats independently,
    are split into `units` ranges and pipelined over three streams: the copy
    of a range's Q, K and V to the device (copy stream), pisa_forward on that
    range (the caller's current stream) and the copy of its O back to the host
    (output stream), so that host-device transfers in both directions overlap
    the computation of other ranges. Each range is one pisa_forward call on a
    shape with batch = planes in the range, heads_q = g, heads_kv = 1; for
    prefill its results equal those of one call on the whole shape bit for bit.
    """

    def __init__(self, shape: Shape, device="cuda", units: int = 8):
        torch = _torch()
        self.shape = shape
        self.device = torch.device(device)
        s = shape
        self.ws = new_workspace(shape, self.device)
        self.q = torch.empty((s.batch, s.heads_q, s.seq_q, s.head_dim), dtype=torch.bfloat16, device=self.device)
        self.k = torch.empty((s.batch, s.heads_kv, s.kv_rows, s.head_dim), dtype=torch.bfloat16, device=self.device)
        self.v = torch.empty_like(self.k)
        self.o = torch.empty_like(self.q)
        self.lse = torch.empty((s.batch, s.heads_q, s.seq_q), dtype=torch.float32, device=self.device)
        planes = s.batch * s.heads_kv
        n = max(1, min(units, planes))
        bounds = [planes * u // n for u in range(n + 1)]
        self.ranges = [(a, b) for a, b in zip(bounds, bounds[1:]) if b > a]
        g = s.heads_q // s.heads_kv
        self.unit_shapes = {b - a: dataclasses.replace(s, batch=b - a, heads_q=g, heads_kv=1) for a, b in self.ranges}
        self.unit_ws = new_workspace(max(self.unit_shapes.values(), key=workspace_size), self.device)
        self.copy_stream = torch.cuda.Stream(self.device)
        self.out_stream = torch.cuda.Stream(self.device)

    def _planes(self, t, per_plane):
        """View of a [B, H, ...] tensor as [planes, per_plane, ...] (planes = B * heads_kv)."""
        return t.view(self.shape.batch * self.shape.heads_kv, per_plane, *t.shape[2:])

    def forward(self, Q, K, V, out=None):
        torch = _torch()
        if Q.is_cuda:
            O, _, _ = forward(self.shape, Q, K, V, self.ws, O=self.o, lse=self.lse)
            return O
        s = self.shape
        g = s.heads_q // s.heads_kv
        if out is None:
            out = torch.empty(tuple(self.o.shape), dtype=self.o.dtype, pin_memory=True)
        hq, hk, hv, ho = self._planes(Q, g), self._planes(K, 1), self._planes(V, 1), self._planes(out, g)
        dq, dk, dv, do = self._planes(self.q, g), self._planes(self.k, 1), self._planes(self.v, 1), self._planes(self.o, g)
        dl = self.lse.view(s.batch * s.heads_kv, g, s.seq_q)
        compute = torch.cuda.current_stream(self.device)
        arrived = []
        # inputs: every range back to back on the copy stream (after earlier work on these buffers)
        self.copy_stream.wait_stream(compute)
        with torch.cuda.stream(self.copy_stream):
            for a, b in self.ranges:
                dq[a:b].copy_(hq[a:b], non_blocking=True)
                dk[a:b].copy_(hk[a:b], non_blocking=True)
                dv[a:b].copy_(hv[a:b], non_blocking=True)
                ev = torch.cuda.Event()
                ev.record(self.copy_stream)
                arrived.append(ev)
        self.out_stream.wait_stream(compute)
        for (a, b), ev in zip(self.ranges, arrived):
            compute.wait_event(ev)
            forward(self.unit_shapes[b - a], dq[a:b], dk[a:b], dv[a:b], self.unit_ws, O=do[a:b], lse=dl[a:b],
                    stream=compute)
            done = torch.cuda.Event()
            done.record(compute)
            self.out_stream.wait_event(done)
            with torch.cuda.stream(self.out_stream):
                ho[a:b].copy_(do[a:b], non_blocking=True)
        compute.wait_stream(self.out_stream)
        return out


# ----------------------------------------------------------------------------- around the attention

# These calls take a few microseconds on the GPU when they serve one token, so their checks are kept
# short: plain comparisons, the error spelled out only when one fails.

def _current_stream(index: int) -> int:
    """The raw current stream of a device (torch's own shortcut to it where it has one: a tenth of the
    microsecond that a Stream object costs)."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _launch(where, call, stream, named, args):
    """call(*args, stream) with the device of the tensors current. `named`: (tensor or None, name); all
    must be on one CUDA device. `stream` must be that device's; None is its current one."""
    torch = _torch()
    dev = named[0][0].get_device()   # (the first is always there)
    for t, name in named:
        if t is not None and t.get_device() != dev or dev < 0:
            if dev < 0 or t.get_device() < 0:
                raise ValueError(f"{name} must be a CUDA tensor")
            raise ValueError(f"{name} must be on cuda:{dev}, got cuda:{t.get_device()}")
    if stream is None:
        raw = _current_stream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"the stream must be one of cuda:{dev}, got {stream.device}")
    else:
        raw = stream.cuda_stream
    if torch.cuda.current_device() == dev:   # kernels launch on the current device
        status = call(*args, raw)
    else:
        with torch.cuda.device(dev):
            status = call(*args, raw)
    if status != OK:
        raise PisaError(status, where)


def _like(t, dtype, shape, name):
    """A contiguous tensor of this type and shape (its device is checked by _launch)."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _rows_like(t, dtype, shape, name):
    """A tensor of this type and shape whose last dim is adjacent; returns its other strides (0 for
    dims of one, whose stride says nothing)."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    a, b, c, last = t.stride()
    if last != 1:
        raise ValueError(f"{name} must have adjacent elements in its last dimension")
    return (a if shape[0] > 1 else 0, b if shape[1] > 1 else 0, c if shape[2] > 1 else 0)


def _status_word(ws):
    torch = _torch()
    if ws.dtype is not torch.uint8 or not ws.is_contiguous() or ws.numel() < 256:
        raise ValueError("ws must be a contiguous uint8 tensor of at least 256 bytes")
    return ws


@dataclasses.dataclass(frozen=True)
class NormRopeShape:
    """Problem description of qk_norm_rope (mirrors pisa_norm_rope_shape; the strides come from the
    tensors of a call)."""
    batch: int
    tokens: int
    heads_q: int
    heads_kv: int
    head_dim: int
    rotary_dim: int
    interleaved: int = 0
    eps: float = 1e-6

    def c(self, xq=(0, 0, 0), xk=(0, 0, 0), dxq=(0, 0, 0), dxk=(0, 0, 0)) -> PisaNormRopeShape:
        structs = self.__dict__.get("_structs")   # one a set of strides, kept by the shape itself
        if structs is None:
            structs = {}
            object.__setattr__(self, "_structs", structs)
        key = (xq, xk, dxq, dxk)
        c = structs.get(key)
        if c is None:
            if len(structs) >= 64:
                structs.clear()
            c = structs[key] = PisaNormRopeShape(
                self.batch, self.tokens, self.heads_q, self.heads_kv, self.head_dim, self.rotary_dim,
                int(self.interleaved), float(self.eps), _i64x3(*xq), _i64x3(*xk), _i64x3(*dxq), _i64x3(*dxk))
        return c


def norm_rope_workspace_size(shape: NormRopeShape) -> int:
    n = ctypes.c_size_t()
    _check(_lib.pisa_norm_rope_workspace_size(ctypes.byref(shape.c()), ctypes.byref(n)),
           "pisa_norm_rope_workspace_size")
    return n.value


def new_norm_rope_workspace(shape: NormRopeShape, device):
    """Workspace of qk_norm_rope_backward (needs no clearing)."""
    torch = _torch()
    return torch.empty(norm_rope_workspace_size(shape), dtype=torch.uint8, device=device)


def _norm_rope_args(s: NormRopeShape, Xq, Xk, pos, inv_freq, wq, wk):
    torch = _torch()
    B, T, D = s.batch, s.tokens, s.head_dim
    sq = _rows_like(Xq, torch.bfloat16, (B, T, s.heads_q, D), "Xq")
    sk = _rows_like(Xk, torch.bfloat16, (B, T, s.heads_kv, D), "Xk")
    f32, half, row = torch.float32, (s.rotary_dim // 2,), (D,)
    for t, name in ((pos, "pos"), (inv_freq, "inv_freq")):
        if t is None and s.rotary_dim:
            raise ValueError(f"{name} is missing")
    if not (pos is None or pos.dtype is torch.int32 and pos.shape == (B, T) and pos.is_contiguous()):
        _like(pos, torch.int32, (B, T), "pos")
    if not (inv_freq is None or inv_freq.dtype is f32 and inv_freq.shape == half and inv_freq.is_contiguous()):
        _like(inv_freq, f32, half, "inv_freq")
    if not (wq is None or wq.dtype is f32 and wq.shape == row and wq.is_contiguous()):
        _like(wq, f32, row, "wq")
    if not (wk is None or wk.dtype is f32 and wk.shape == row and wk.is_contiguous()):
        _like(wk, f32, row, "wk")
    return sq, sk


def qk_norm_rope(shape: NormRopeShape, Xq, Xk, pos, inv_freq, wq=None, wk=None, Q=None, K=None, stream=None):
    """RMS norm of every head of Xq [B, T, heads_q, D] and Xk [B, T, heads_kv, D] (bf16, any strides:
    views into a packed projection) with weights wq, wk (fp32 [D], None = ones), and rotation of its
    first rotary_dim dims by pos (int32 [B, T]) times inv_freq (fp32 [rotary_dim / 2]). Returns Q
    [B, heads_q, T, D] and K [B, heads_kv, T, D], the attention's layout."""
    torch = _torch()
    s = shape
    sq, sk = _norm_rope_args(s, Xq, Xk, pos, inv_freq, wq, wk)
    qs, ks = (s.batch, s.heads_q, s.tokens, s.head_dim), (s.batch, s.heads_kv, s.tokens, s.head_dim)
    Q = _made(stream, lambda: Xq.new_empty(qs)) if Q is None else _like(Q, torch.bfloat16, qs, "Q")
    K = _made(stream, lambda: Xq.new_empty(ks)) if K is None else _like(K, torch.bfloat16, ks, "K")
    _launch("pisa_qk_norm_rope", _lib.pisa_qk_norm_rope, stream,
            ((Xq, "Xq"), (Xk, "Xk"), (pos, "pos"), (inv_freq, "inv_freq"), (wq, "wq"), (wk, "wk"), (Q, "Q"), (K, "K")),
            (s.c(sq, sk), Xq.data_ptr(), Xk.data_ptr(), _ptr(wq), _ptr(wk), _ptr(inv_freq), _ptr(pos), Q.data_ptr(),
             K.data_ptr()))
    return Q, K


def qk_norm_rope_backward(shape: NormRopeShape, Xq, Xk, pos, inv_freq, dQ, dK, wq=None, wk=None, ws=None, dXq=None,
                          dXk=None, stream=None):
    """Gradients of qk_norm_rope for dQ [B, heads_q, T, D] and dK: (dXq, dXk, dwq, dwk). dXq and dXk
    (the shapes of Xq and Xk; new contiguous tensors if None) may be views into a packed gradient.
    dwq, dwk: fp32 [D], None where the weight is None."""
    torch = _torch()
    s = shape
    B, T, D = s.batch, s.tokens, s.head_dim
    sq, sk = _norm_rope_args(s, Xq, Xk, pos, inv_freq, wq, wk)
    _like(dQ, torch.bfloat16, (B, s.heads_q, T, D), "dQ")
    _like(dK, torch.bfloat16, (B, s.heads_kv, T, D), "dK")
    dXq = _made(stream, lambda: Xq.new_empty((B, T, s.heads_q, D))) if dXq is None else dXq
    dXk = _made(stream, lambda: Xq.new_empty((B, T, s.heads_kv, D))) if dXk is None else dXk
    gq = _rows_like(dXq, torch.bfloat16, (B, T, s.heads_q, D), "dXq")
    gk = _rows_like(dXk, torch.bfloat16, (B, T, s.heads_kv, D), "dXk")
    dwq = _made(stream, lambda: wq.new_empty(D)) if wq is not None else None
    dwk = _made(stream, lambda: wk.new_empty(D)) if wk is not None else None
    if ws is None:
        ws = _made(stream, lambda: new_norm_rope_workspace(s, Xq.device))
    elif not ws.is_contiguous():   # its bytes are counted from its elements
        raise ValueError("ws must be contiguous")
    _launch("pisa_qk_norm_rope_backward", _lib.pisa_qk_norm_rope_backward, stream,
            ((Xq, "Xq"), (Xk, "Xk"), (pos, "pos"), (inv_freq, "inv_freq"), (wq, "wq"), (wk, "wk"), (dQ, "dQ"),
             (dK, "dK"), (dXq, "dXq"), (dXk, "dXk"), (ws, "ws")),
            (s.c(sq, sk, gq, gk), Xq.data_ptr(), Xk.data_ptr(), _ptr(wq), _ptr(wk), _ptr(inv_freq), _ptr(pos),
             dQ.data_ptr(), dK.data_ptr(), dXq.data_ptr(), dXk.data_ptr(), _ptr(dwq), _ptr(dwk), ws.data_ptr(),
             ws.numel() * ws.element_size()))
    return dXq, dXk, dwq, dwk


@dataclasses.dataclass(frozen=True)
class CacheShape:
    """Problem description of a K/V cache (mirrors pisa_cache_shape)."""
    batch: int
    heads_kv: int
    capacity: int
    head_dim: int
    format: int = CACHE_E4M3

    def c(self) -> PisaCacheShape:
        return PisaCacheShape(self.batch, self.heads_kv, self.capacity, self.head_dim, int(self.format))


class Cache:
    """A K/V cache's buffers: k and v [B, heads_kv, capacity, D] (bf16, or float8_e4m3fn with the
    exponent bytes k_exp and v_exp, uint8 [B, heads_kv, capacity], 1 .. 255: a row is its values times
    2^(byte - 127), or NaN for 255). v and v_exp may be None for calls that only read keys (cache_append_pyramid).
    The buffers are those of its making (a larger cache is a new Cache); every call checks that they
    are still such buffers and takes their addresses as they are then."""

    def __init__(self, shape: CacheShape, k, v, k_exp=None, v_exp=None):
        if v is None and v_exp is not None:
            raise ValueError("v_exp without v")
        self._shape, self._c, self._buffers = shape, shape.c(), (k, v, k_exp, v_exp)
        torch = _torch()
        self._rows = torch.Size((shape.batch, shape.heads_kv, shape.capacity))
        self._whole = torch.Size((*self._rows, shape.head_dim))
        self._types = (torch.float8_e4m3fn if shape.format == CACHE_E4M3 else torch.bfloat16, torch.uint8)
        self._check()

    def _check(self):
        dt, u8 = self._types
        k, v, k_exp, v_exp = self._buffers
        fp8 = self._shape.format == CACHE_E4M3
        for t, e, name in ((k, k_exp, "k"), (v, v_exp, "v")):
            if t is None and name == "v":
                continue
            _like(t, dt, self._whole, name)
            if fp8:
                if e is None:
                    raise ValueError(f"{name}_exp is missing")
                _like(e, u8, self._rows, f"{name}_exp")
            elif e is not None:
                raise ValueError(f"{name}_exp belongs to an e4m3 cache")
        for t, name in ((v, "v"), (k_exp, "k_exp"), (v_exp, "v_exp")):
            if t is not None and t.device != k.device:
                raise ValueError(f"{name} must be on {k.device}, got {t.device}")

    shape = property(lambda self: self._shape)
    k = property(lambda self: self._buffers[0])
    v = property(lambda self: self._buffers[1])
    k_exp = property(lambda self: self._buffers[2])
    v_exp = property(lambda self: self._buffers[3])
    device = property(lambda self: self._buffers[0].device)

    def _both(self):
        if self._buffers[1] is None:
            raise ValueError("the cache has no v")
        return self

    def _ptrs(self):
        """The buffers' addresses at this call; what a resize_ or set_ made of them is checked first."""
        k, v, k_exp, v_exp = self._buffers
        dt, u8 = self._types
        whole, rows, dev = self._whole, self._rows, k.get_device()
        if not (k.dtype is dt and k.shape == whole and k.is_contiguous() and
                (v is None or v.dtype is dt and v.shape == whole and v.is_contiguous() and v.get_device() == dev)):
            self._check()
        if k_exp is None:
            return k.data_ptr(), _ptr(v), None, None
        if not (k_exp.dtype is u8 and k_exp.shape == rows and k_exp.is_contiguous() and k_exp.get_device() == dev and
                (v_exp is None or v_exp.dtype is u8 and v_exp.shape == rows and v_exp.is_contiguous() and
                 v_exp.get_device() == dev)):
            self._check()
        return k.data_ptr(), _ptr(v), k_exp.data_ptr(), _ptr(v_exp)


def new_cache(shape: CacheShape, device) -> Cache:
    """A cache whose rows are all zero."""
    torch = _torch()
    s = shape
    fp8 = s.format == CACHE_E4M3
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    k, v = (torch.zeros((s.batch, s.heads_kv, s.capacity, s.head_dim), dtype=dt, device=device) for _ in range(2))
    ke, ve = (torch.ones((s.batch, s.heads_kv, s.capacity), dtype=torch.uint8, device=device) if fp8 else None
              for _ in range(2))
    return Cache(s, k, v, ke, ve)


def new_cache_workspace(device):
    """A status word for cache_write and cache_read (any other workspace serves as well)."""
    torch = _torch()
    return torch.zeros(256, dtype=torch.uint8, device=device)


def _ranges(B, start, count):
    torch = _torch()
    for t, name in ((start, "start"), (count, "count")):
        if t is not None:
            _like(t, torch.int32, (B,), name)


def cache_write(cache: Cache, K, V, ws, start=None, count=None, stream=None) -> None:
    """Writes the rows of K and V (bf16 [B, heads_kv, tokens, D], any strides) to the positions
    start[b] + t, t < count[b] (int32 [B] on the device; 0 and all rows if None), quantising them if
    the cache is e4m3. A sequence whose rows do not fit is left alone and recorded in ws."""
    torch = _torch()
    s = cache._both().shape
    rows = (s.batch, s.heads_kv, K.shape[2] if K.dim() == 4 else -1, s.head_dim)
    sk, sv = _rows_like(K, torch.bfloat16, rows, "K"), _rows_like(V, torch.bfloat16, rows, "V")
    _ranges(s.batch, start, count)
    _status_word(ws)
    _launch("pisa_cache_write", _lib.pisa_cache_write, stream,
            ((cache.k, "cache"), (K, "K"), (V, "V"), (start, "start"), (count, "count"), (ws, "ws")),
            (cache._c, rows[2], K.data_ptr(), V.data_ptr(), _i64x3(*sk), _i64x3(*sv), _ptr(start), _ptr(count),
             *cache._ptrs(), ws.data_ptr()))


def cache_read(cache: Cache, tokens: int, ws, start=None, count=None, K=None, V=None, stream=None):
    """The rows start[b] + t, t < count[b], of K and V as bf16 [B, heads_kv, tokens, D]. Rows that do
    not count keep what K and V held (zeros in new tensors)."""
    torch = _torch()
    s = cache._both().shape
    rows = (s.batch, s.heads_kv, int(tokens), s.head_dim)
    if tokens < 1:
        raise ValueError("tokens must be at least 1")
    fill = torch.empty if count is None and start is None else torch.zeros

    def make():
        return fill(rows, dtype=torch.bfloat16, device=cache.device)

    K = _made(stream, make) if K is None else _like(K, torch.bfloat16, rows, "K")
    V = _made(stream, make) if V is None else _like(V, torch.bfloat16, rows, "V")
    _ranges(s.batch, start, count)
    _status_word(ws)
    _launch("pisa_cache_read", _lib.pisa_cache_read, stream,
            ((cache.k, "cache"), (K, "K"), (V, "V"), (start, "start"), (count, "count"), (ws, "ws")),
            (cache._c, rows[2], *cache._ptrs(), _ptr(start), _ptr(count), K.data_ptr(), V.data_ptr(), ws.data_ptr()))
    return K, V


def cache_append_pyramid(shape: Shape, cache: Cache, pyramid, seq_kv_old: int, stream=None):
    """append_pyramid for an e4m3 cache: brings `pyramid` (fp32 [B, heads_kv, nodes, D], that of the
    cache at length seq_kv_old; zeros for 0) up to shape.seq_kv."""
    torch = _torch()
    s = cache.shape
    if s.format != CACHE_E4M3:
        raise ValueError("cache_append_pyramid takes an e4m3 cache (append_pyramid a bf16 one)")
    if (s.batch, s.heads_kv, s.capacity, s.head_dim) != (shape.batch, shape.heads_kv, shape.kv_rows, shape.head_dim):
        raise ValueError("the shape's batch, heads_kv, capacity and head_dim must be the cache's")
    _like(pyramid, torch.float32, (s.batch, s.heads_kv, shape.n_nodes, s.head_dim), "pyramid")
    k, _, k_exp, _ = cache._ptrs()
    _launch("pisa_cache_append_pyramid", _lib.pisa_cache_append_pyramid, stream,
            ((cache.k, "cache"), (pyramid, "pyramid")), (shape.c(), k, k_exp, pyramid.data_ptr(), int(seq_kv_old)))
    return pyramid


@dataclasses.dataclass(frozen=True)
class TreeShape:
    """Problem description of tree_attention (mirrors pisa_tree_shape)."""
    batch: int
    heads_q: int
    heads_kv: int
    drafts: int
    capacity: int
    head_dim: int
    format: int = CACHE_E4M3
    block: int = 64
    seq_kv: int = 0
    topk: int = 0
    select_per_qhead: int = 0
    scale: float = 0.0

    def c(self) -> PisaTreeShape:
        c = self.__dict__.get("_struct")   # kept by the shape itself
        if c is None:
            c = PisaTreeShape(self.batch, self.heads_q, self.heads_kv, self.drafts, self.capacity, self.head_dim,
                              int(self.format), self.block, self.seq_kv, self.topk, int(self.select_per_qhead),
                              float(self.scale))
            object.__setattr__(self, "_struct", c)
        return c

    @property
    def hsel(self) -> int:
        return self.heads_q if self.select_per_qhead else self.heads_kv


def tree_workspace_size(shape: TreeShape) -> int:
    n = ctypes.c_size_t()
    _check(_lib.pisa_tree_workspace_size(ctypes.byref(shape.c()), ctypes.byref(n)), "pisa_tree_workspace_size")
    return n.value


def new_tree_workspace(shape: TreeShape, device):
    """Workspace of tree_attention with a cleared status word."""
    torch = _torch()
    ws = torch.empty(tree_workspace_size(shape), dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def tree_attention(shape: TreeShape, cache: Cache, Q, K, V, mask, cache_len, ws, idx=None, O=None, lse=True,
                   stream=None):
    """Attention of the drafted tokens Q [B, heads_q, T, D] over the cache's first cache_len[b] rows
    (int32 [B]; those of the blocks of idx [B, Hsel, 1, topk] and from seq_kv on, or all) and over the
    drafted K, V [B, heads_kv, T, D] whose bits are set in mask (int64 [B, T], bit j of token t's word
    = token t attends drafted token j). Returns (O, lse)."""
    torch = _torch()
    s, c = shape, cache._both().shape
    B, Hq, Hkv, T, D = s.batch, s.heads_q, s.heads_kv, s.drafts, s.head_dim
    if (c.batch, c.heads_kv, c.capacity, c.head_dim, c.format) != (B, Hkv, s.capacity, D, s.format):
        raise ValueError("the shape's batch, heads_kv, capacity, head_dim and format must be the cache's")
    qs, kvs, bf16 = (B, Hq, T, D), (B, Hkv, T, D), torch.bfloat16
    if not (Q.dtype is bf16 and K.dtype is bf16 and V.dtype is bf16 and mask.dtype is torch.int64 and
            cache_len.dtype is torch.int32 and Q.shape == qs and K.shape == kvs and V.shape == kvs and
            mask.shape == (B, T) and cache_len.shape == (B,) and Q.is_contiguous() and K.is_contiguous() and
            V.is_contiguous() and mask.is_contiguous() and cache_len.is_contiguous()):
        _like(Q, bf16, qs, "Q")
        _like(K, bf16, kvs, "K")
        _like(V, bf16, kvs, "V")
        _like(mask, torch.int64, (B, T), "mask")
        _like(cache_len, torch.int32, (B,), "cache_len")
    if (idx is not None) != (s.topk > 0):
        raise ValueError("idx goes with topk > 0")
    if idx is not None:
        _like(idx, torch.int32, (B, s.hsel, 1, s.topk), "idx")
    O = _made(stream, lambda: torch.empty_like(Q)) if O is None else _like(O, bf16, qs, "O")
    if lse is True:
        lse = _made(stream, lambda: Q.new_empty((B, Hq, T), dtype=torch.float32))
    elif lse is False:
        lse = None
    elif lse is not None:
        _like(lse, torch.float32, (B, Hq, T), "lse")
    _status_word(ws)
    _launch("pisa_tree_attention", _lib.pisa_tree_attention, stream,
            ((Q, "Q"), (K, "K"), (V, "V"), (mask, "mask"), (cache_len, "cache_len"), (cache.k, "cache"), (idx, "idx"),
             (O, "O"), (lse, "lse"), (ws, "ws")),
            (s.c(), Q.data_ptr(), K.data_ptr(), V.data_ptr(), mask.data_ptr(), *cache._ptrs(), cache_len.data_ptr(),
             _ptr(idx), O.data_ptr(), _ptr(lse), ws.data_ptr(), ws.numel()))
    return O, lse


# ----------------------------------------------------------------------------- measurement helpers

def attention_pairs(idx: np.ndarray, shape: Shape) -> int:
    """Unmasked (query, key) pairs the attention evaluates for a selection (host arithmetic).

    A selected block j < i contributes b*b pairs per query head, the diagonal
    block (causal) b(b+1)/2; decode contributes b per selected block per head.
    """
    b = shape.block
    heads_per_row = 1 if shape.select_per_qhead else shape.heads_q // shape.heads_kv
    valid = idx >= 0
    if shape.decode:
        return int(valid.sum()) * b * heads_per_row
    full = int(valid.sum()) * b * b
    if shape.causal:
        i = np.arange(idx.shape[2]).reshape(1, 1, -1, 1)
        diag = int(((idx == i) & valid).sum())
        full -= diag * (b * b - b * (b + 1) // 2)
    return full * heads_per_row


def attention_flops(idx: np.ndarray, shape: Shape) -> float:
    """Algorithmic FLOPs of the attention step: 4 * D per unmasked (query, key) pair (QK^T and PV)."""
    return 4.0 * shape.head_dim * attention_pairs(idx, shape)


def default_scale(shape: Shape) -> float:
    return shape.scale if shape.scale > 0 else 1.0 / math.sqrt(shape.head_dim)
