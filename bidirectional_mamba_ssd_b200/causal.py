"""Serving with the forward scan alone: prompts, single tokens and the pages of
the pool of states they share (include/ssd_bidir.h: ssd_causal_fwd,
ssd_causal_step, ssd_cache_copy, ssd_cache_compact).

  states (slots, H, P, N) fp32     a pool; one per layer, or (layers, slots, H, P, N) for the page calls
  x (batch, L, H, P), dt (batch, L, H), B, C (batch, L, G, N); A, D, dt_bias (H) fp32
  a single token drops the L dimension

x, dt, B and C may be views in batch and token (the slices of one projection);
their last two dimensions (dt: its last) are contiguous.

Calls without a workspace of their own use the stream's, or, while a CUDA graph
is being captured, one that belongs to the graph: two graphs never share one.
"""
from __future__ import annotations

import torch

from . import (SSD_OP_CAUSAL_FWD, SSD_OP_CAUSAL_STEP, SSD_PATH_AUTO, Workspace, _check, _DT, _need, _workspace, lib)

_INF = float("inf")


def _rows(t, name, dtype, device, shape):
    """t has this shape, its dimensions past batch (and token) contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)} (got {tuple(t.shape)})")


def _inner(t, name, dims):
    """The last `dims` dimensions of t are contiguous."""
    st, sh = t.stride(), t.shape
    if (sh[-1] > 1 and st[-1] != 1) or (dims == 2 and sh[-2] > 1 and st[-2] != sh[-1]):
        raise ValueError(f"{name}: the last {dims} dimensions must be contiguous (strides {st})")


def _vector(t, name, dtype, device, n):
    if t is None:
        return 0
    _need(t, name, dtype, device, 1)
    if t.shape[0] != n:
        raise ValueError(f"{name} must have {n} entries (got {t.shape[0]})")
    return t.data_ptr()


def _pool(t, name, device, rows, H, P, N):
    """A pool of states with `rows` pages (None: any number)."""
    _need(t, name, torch.float32, device, 4)
    if t.shape[1:] != (H, P, N) or (rows is not None and t.shape[0] != rows):
        raise ValueError(f"{name} must be ({'slots' if rows is None else rows}, {H}, {P}, {N}) (got {tuple(t.shape)})")


def _apart(a, b, na, nb):
    """The same array, or no byte in common."""
    pa, pb = a.data_ptr(), b.data_ptr()
    if pa != pb and pa < pb + b.numel() * b.element_size() and pb < pa + a.numel() * a.element_size():
        raise ValueError(f"{na} and {nb} overlap without being the same array")


class _On:
    """The tensors' device as the current one, where it is not already."""

    def __init__(self, device):
        self.guard = None if device.index == torch.cuda.current_device() else torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _scratch(device, stream, workspace):
    """The workspace of a call: the caller's, the graph's being captured, or the stream's."""
    if workspace is None and torch.cuda.is_current_stream_capturing():
        return Workspace(device)
    if workspace is not None and workspace.device.index not in (None, device.index):
        raise ValueError(f"workspace is on {workspace.device}, expected {device}")
    return _workspace(device, stream, workspace)


def ssd_causal_fwd(x, dt, A, B, C, D=None, init=None, *, seqlens=None, slots=None, dt_bias=None, dt_min: float = 0.0,
                   dt_max: float = _INF, out=None, state_out=None, path: int = SSD_PATH_AUTO,
                   workspace: Workspace | None = None):
    """The forward scan over prompts with its outputs (include/ssd_bidir.h:
    ssd_causal_fwd): returns (out like x, end states).

    seqlens (batch) int32: tokens of each sequence; outputs behind them are zero.
    init: start states, (batch, H, P, N), or with slots (batch) int32 a pool
    (nslots, H, P, N) whose page slots[b] is row b's; None starts from zero.
    state_out: where the end states go, laid out as init; with slots it
    defaults to init (in place). dt_bias (H): dt is the raw projection."""
    _need_cuda(x, "x", 4)
    dev, io = x.device, x.dtype
    if io not in _DT:
        raise ValueError(f"x dtype {io} not supported (float32 or bfloat16)")
    batch, L, H, P = x.shape
    if not isinstance(B, torch.Tensor) or B.dim() != 4:
        raise ValueError("B must be (batch, L, G, N)")
    G, N = B.shape[2:]
    _rows(dt, "dt", io, dev, (batch, L, H))
    _rows(B, "B", io, dev, (batch, L, G, N))
    _rows(C, "C", io, dev, (batch, L, G, N))
    for t, name, dims in ((x, "x", 2), (dt, "dt", 1), (B, "B", 2), (C, "C", 2)):
        _inner(t, name, dims)
    if A is None:
        raise ValueError("A is required")
    pa, pd, pb = (_vector(t, n, torch.float32, dev, H) for t, n in ((A, "A"), (D, "D"), (dt_bias, "dt_bias")))
    plen, pslot = (_vector(t, n, torch.int32, dev, batch) for t, n in ((seqlens, "seqlens"), (slots, "slots")))
    rows = batch
    if slots is not None:
        if state_out is None:
            state_out = init
        if state_out is None:
            raise ValueError("slots need a pool: init, state_out or both")
        rows = state_out.shape[0]
    elif state_out is None:
        state_out = torch.empty(batch, H, P, N, dtype=torch.float32, device=dev)
    _pool(state_out, "state_out", dev, rows, H, P, N)
    if init is not None and init is not state_out:
        _pool(init, "init", dev, rows, H, P, N)
        _apart(init, state_out, "init", "state_out")
    if out is None:
        out = torch.empty((batch, L, H, P), dtype=io, device=dev)
    else:
        _need(out, "out", io, dev, 4)
        if out.shape != x.shape:
            raise ValueError("out must have x's shape")
    xs, ds, bs, cs = x.stride(), dt.stride(), B.stride(), C.stride()
    with _On(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        ws = _scratch(dev, stream, workspace)
        nbytes = lib.ssd_workspace_bytes(SSD_OP_CAUSAL_FWD, batch, L, H, P, N, G, 0, _DT[io])
        with ws.lock:
            buf = ws.get(nbytes)
            rc = lib.ssd_causal_fwd(x.data_ptr(), dt.data_ptr(), pa, B.data_ptr(), C.data_ptr(), pd, pb, dt_min, dt_max,
                                    plen, pslot, init.data_ptr() if init is not None else 0, state_out.data_ptr(),
                                    out.data_ptr(), xs[0], xs[1], ds[0], ds[1], bs[0], bs[1], cs[0], cs[1], rows,
                                    batch, L, H, P, N, G, _DT[io], path, buf.data_ptr(), buf.numel(), stream)
    _check(rc, "ssd_causal_fwd")
    return out, state_out


def ssd_causal_step(x, dt, A, B, C, D, states, slots=None, *, dt_bias=None, dt_min: float = 0.0, dt_max: float = _INF,
                    out=None, state_out=None, workspace: Workspace | None = None):
    """One token of every row (include/ssd_bidir.h: ssd_causal_step): x (batch, H,
    P), dt (batch, H), B, C (batch, G, N), D (H) or None. The states, (batch, H,
    P, N) or with slots (batch) int32 a pool of pages, advance in place unless
    state_out is given. Returns out like x."""
    _need_cuda(x, "x", 3)
    dev, io = x.device, x.dtype
    if io not in _DT:
        raise ValueError(f"x dtype {io} not supported (float32 or bfloat16)")
    batch, H, P = x.shape
    if not isinstance(B, torch.Tensor) or B.dim() != 3:
        raise ValueError("B must be (batch, G, N)")
    G, N = B.shape[1:]
    _rows(dt, "dt", io, dev, (batch, H))
    _rows(B, "B", io, dev, (batch, G, N))
    _rows(C, "C", io, dev, (batch, G, N))
    for t, name, dims in ((x, "x", 2), (dt, "dt", 1), (B, "B", 2), (C, "C", 2)):
        _inner(t, name, dims)
    if A is None:
        raise ValueError("A is required")
    pa, pd, pb = (_vector(t, n, torch.float32, dev, H) for t, n in ((A, "A"), (D, "D"), (dt_bias, "dt_bias")))
    pslot = _vector(slots, "slots", torch.int32, dev, batch)
    _pool(states, "states", dev, batch if slots is None else None, H, P, N)
    if state_out is None:
        state_out = states
    elif state_out is not states:
        _pool(state_out, "state_out", dev, states.shape[0], H, P, N)
        _apart(states, state_out, "states", "state_out")
    if out is None:
        out = torch.empty((batch, H, P), dtype=io, device=dev)
    else:
        _need(out, "out", io, dev, 3)
        if out.shape != x.shape:
            raise ValueError("out must have x's shape")
    with _On(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        pws = nws = 0
        if slots is not None:
            ws = _scratch(dev, stream, workspace)
            nbytes = 256 if batch <= 2048 else lib.ssd_workspace_bytes(SSD_OP_CAUSAL_STEP, batch, 1, H, P, N, G, 0, _DT[io])
            ws.lock.acquire()
            buf = ws.get(nbytes)
            pws, nws = buf.data_ptr(), buf.numel()
        try:
            rc = lib.ssd_causal_step(x.data_ptr(), dt.data_ptr(), pa, B.data_ptr(), C.data_ptr(), pd, pb, dt_min, dt_max,
                                     pslot, states.data_ptr(), state_out.data_ptr(), out.data_ptr(), x.stride(0),
                                     dt.stride(0), B.stride(0), C.stride(0), states.shape[0], batch, H, P, N, G,
                                     _DT[io], pws, nws, stream)
        finally:
            if slots is not None:
                ws.lock.release()
    _check(rc, "ssd_causal_step")
    return out


def _need_cuda(t, name, ndim):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims (got {tuple(t.shape)})")


def _pages(pool):
    _need(pool, "pool")
    if pool.dim() < 3:
        raise ValueError(f"pool must be (layers, slots, page...) (got {tuple(pool.shape)})")
    layers, nslots = pool.shape[:2]
    page = pool.element_size()
    for n in pool.shape[2:]:
        page *= n
    return layers, nslots, page


def ssd_cache_copy(pool, src, dst, *, workspace: Workspace | None = None):
    """Pages of a pool (layers, slots, ...) of any dtype, in place and in every
    layer: page dst[i] <- page src[i], or zero where src[i] is -1, in the order
    of i (include/ssd_bidir.h: ssd_cache_copy). src, dst (n) int32. Returns pool."""
    layers, nslots, page = _pages(pool)
    dev = pool.device
    n = src.shape[0] if isinstance(src, torch.Tensor) and src.dim() == 1 else 0
    if src is None or dst is None:
        raise ValueError("src and dst are required")
    ps, pd = _vector(src, "src", torch.int32, dev, n), _vector(dst, "dst", torch.int32, dev, n)
    with _On(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        ws = _scratch(dev, stream, workspace)
        with ws.lock:
            buf = ws.get(256)
            rc = lib.ssd_cache_copy(pool.data_ptr(), page, layers, nslots, ps, pd, n, buf.data_ptr(), buf.numel(), stream)
    _check(rc, "ssd_cache_copy")
    return pool


def ssd_cache_compact(pool, table, *, workspace: Workspace | None = None):
    """Move the pages that table (rows) int32 names (-1: none) to the front of a
    pool (layers, slots, ...), in place, with the fewest moves (include/
    ssd_bidir.h: ssd_cache_compact). Returns (the table that goes with the moved
    pages, the number of live pages as an int32 tensor of one)."""
    layers, nslots, page = _pages(pool)
    dev = pool.device
    _need(table, "table", torch.int32, dev, 1)
    new = torch.empty_like(table)
    live = torch.empty(1, dtype=torch.int32, device=dev)
    with _On(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        ws = _scratch(dev, stream, workspace)
        with ws.lock:
            buf = ws.get(256)
            rc = lib.ssd_cache_compact(pool.data_ptr(), page, layers, nslots, table.data_ptr(), table.shape[0],
                                       new.data_ptr(), live.data_ptr(), buf.data_ptr(), buf.numel(), stream)
    _check(rc, "ssd_cache_compact")
    return new, live
