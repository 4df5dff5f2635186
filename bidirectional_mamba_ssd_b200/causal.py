"""Serving with the forward scan alone: prompts, single tokens and the pages of
the pool of states they share (include/ssd_bidir.h: ssd_causal_fwd,
ssd_causal_step, ssd_cache_copy, ssd_cache_compact).

  states (slots, H, P, N) fp32     a pool; one per layer, or (layers, slots, H, P, N) for the page calls
  x (batch, L, H, P), dt (batch, L, H), B, C (batch, L, G, N); A, D, dt_bias (H) fp32
  a single token drops the L dimension

x, dt, B and C may be views in batch and token (the slices of one projection);
their last two dimensions (dt: its last) are contiguous.

Calls without a workspace of their own use the stream's. While a CUDA graph is
being captured they use scratch that belongs to the graph (two graphs never share
any), and what they report at a replay, on whatever stream, ssd_get_device_status()
reads from the library's own header of the device. A workspace of the caller's works
under capture too; it is to have its size before (a call outside the capture gives
it that), and its own status() has what is reported.

A single token's kernel takes a few microseconds, less than ctypes takes to call it. So
each function first offers its arguments to csrc/ssd_binding.cpp, which makes the
call if all of them are as they should be; what follows here is for the calls that it
leaves alone: bad arguments (their messages), another device than the current one,
a workspace that has yet to be made or to grow, and a graph's own under capture. Where
that extension is missing or built for another torch, every call takes this way.
"""
from __future__ import annotations

import ctypes
import functools
import threading
import warnings

import torch

from . import (SSD_OP_CAUSAL_FWD, SSD_OP_CAUSAL_STEP, SSD_PATH_AUTO, Workspace, _captured, _captured_header, _check,
               _default_ws, _DT, _workspace, lib)


class _Absent:
    """In the extension's place where it is missing or unfit: leaves every call to this module."""
    causal_fwd = causal_step = cache_copy = cache_compact = staticmethod(lambda *a: NotImplemented)


def _load_binding():
    try:
        from . import _binding as b
        if b.torch_version != str(torch.__version__):
            raise ImportError(f"built for torch {b.torch_version}, this is {torch.__version__}")
        entries = (lib.ssd_causal_fwd, lib.ssd_causal_step, lib.ssd_cache_copy, lib.ssd_cache_compact)
        b.setup(*(ctypes.cast(f, ctypes.c_void_p).value for f in entries), _default_ws, _check)
        return b
    except (ImportError, AttributeError) as e:
        warnings.warn(f"the C++ part of the serving calls' binding is not used, calls take longer on the host ({e}); "
                      "it is built by `python -c 'import __graft_entry__ as g; g.build()'`", RuntimeWarning, stacklevel=2)
        return _Absent


_binding = _load_binding()

_INF = float("inf")
_INT = 2**31 - 1
_HEADER = 256          # bytes of a workspace's status header
_F32, _I32 = torch.float32, torch.int32
_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream
_capturing = torch._C._cuda_isCurrentStreamCapturing


@functools.lru_cache(maxsize=4096)
def _bytes(device, op, batch, L, H, P, N, G, code):
    """ssd_workspace_bytes on a device (whose SM count it goes by)."""
    return lib.ssd_workspace_bytes(op, batch, L, H, P, N, G, 0, code)


def _fail(t, name, dtype, dev, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev or dev.type != "cuda":
        raise ValueError(f"{name} is on {t.device}, expected {dev if dev.type == 'cuda' else 'a CUDA device'}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)} (got {tuple(t.shape)})")
    raise ValueError(f"{name}: the dimensions past batch and token must be contiguous (shape {tuple(t.shape)}, "
                     f"strides {t.stride()})")


def _rows(t, name, dtype, dev, shape, dims):
    """The strides of t, which has this shape and its last `dims` dimensions contiguous."""
    try:
        if t.dtype is dtype and t.device == dev and t.shape == shape:
            st = t.stride()
            if (st[-1] == 1 or shape[-1] <= 1) and (dims == 1 or st[-2] == shape[-1] or shape[-2] <= 1):
                return st
    except (AttributeError, IndexError):
        pass
    _fail(t, name, dtype, dev, shape)


def _whole(t, name, dtype, dev, shape):
    """The address of t, contiguous and of this shape; 0 for None."""
    if t is None:
        return 0
    try:
        if t.dtype is dtype and t.device == dev and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _fail(t, name, dtype, dev, shape)


def _lead(t, name, ndim):
    """Device, I/O type and shape of the tensor that the others are checked against."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (got {dev})")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims (got {tuple(t.shape)})")
    return dev, t.dtype, t.shape


def _states(t, name, dev, slots, rows, page):
    """The number of pages of a pool: one a row, or any number where slots name them."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    n = t.shape[0] if slots is not None and t.dim() > 0 else rows
    _whole(t, name, _F32, dev, (n, *page))
    return n


def _apart(a, b, na, nb):
    """The same array, or no byte in common."""
    pa, pb, n = a.data_ptr(), b.data_ptr(), 4 * a.numel()
    if pa != pb and pa < pb + n and pb < pa + n:
        raise ValueError(f"{na} and {nb} overlap without being the same array")


class _Captured:
    """The workspace of one call that is being captured: the library's own header where the call needs no more, else memory
    of the graph's pool, which a node of the graph prepares."""

    def __init__(self, dev, stream):
        self.dev, self.stream, self.lock = dev, stream, threading.Lock()
        _captured.add(dev.index)

    def get(self, nbytes):
        if nbytes <= _HEADER:
            return _Header(_captured_header())
        buf = torch.empty(nbytes, dtype=torch.uint8, device=self.dev)
        _check(lib.ssd_workspace_init_captured(buf.data_ptr(), nbytes, self.stream), "ssd_workspace_init_captured")
        return buf


class _Header:
    """The library's own status header, as far as a call looks at a buffer."""

    def __init__(self, address):
        self.address = address

    def data_ptr(self):
        return self.address

    def numel(self):
        return _HEADER


def _scratch(dev, stream, workspace):
    """The workspace of a call: the caller's, the graph's being captured, or the stream's."""
    if workspace is None:
        return _Captured(dev, stream) if _capturing() else _workspace(dev, stream, None)
    if workspace.device.index not in (None, dev.index):
        raise ValueError(f"workspace is on {workspace.device}, expected {dev}")
    return workspace


def ssd_causal_fwd(x, dt, A, B, C, D=None, init=None, *, seqlens=None, slots=None, dt_bias=None, dt_min: float = 0.0,
                   dt_max: float = _INF, out=None, state_out=None, path: int = SSD_PATH_AUTO,
                   workspace: Workspace | None = None):
    """The forward scan over prompts with its outputs (include/ssd_bidir.h:
    ssd_causal_fwd): returns (out like x, end states).

    seqlens (batch) int32: tokens of each sequence; outputs behind them are zero.
    init: start states, (batch, H, P, N), or with slots (batch) int32 a pool
    (nslots, H, P, N) whose page slots[b] is row b's; None starts from zero.
    state_out: where the end states go, laid out as init; with slots it
    defaults to init (in place). dt_bias (H): dt is the raw projection.
    path: SSD_PATH_AUTO takes bf16 inputs to the tensor cores, which round the
    masked C.B^T tile and the copy of the state that outputs read to bf16 (end
    states keep fp32 accuracy); SSD_PATH_SIMT rounds nothing but the output."""
    got = _binding.causal_fwd(x, dt, A, B, C, D, init, seqlens, slots, dt_bias, dt_min, dt_max, out, state_out, path,
                              workspace)
    if got is not NotImplemented:
        return got
    dev, io, xshape = _lead(x, "x", 4)
    if dev.index != _device():
        with torch.cuda.device(dev):
            return ssd_causal_fwd(x, dt, A, B, C, D, init, seqlens=seqlens, slots=slots, dt_bias=dt_bias, dt_min=dt_min,
                                  dt_max=dt_max, out=out, state_out=state_out, path=path, workspace=workspace)
    code = _DT.get(io)
    if code is None:
        raise ValueError(f"x dtype {io} not supported (float32 or bfloat16)")
    batch, L, H, P = xshape
    G, N = B.shape[2:] if isinstance(B, torch.Tensor) and B.dim() == 4 else (0, 0)
    bc, vec, row = (batch, L, G, N), (H,), (batch,)
    xs, ds = _rows(x, "x", io, dev, xshape, 2), _rows(dt, "dt", io, dev, (batch, L, H), 1)
    bs, cs = _rows(B, "B", io, dev, bc, 2), _rows(C, "C", io, dev, bc, 2)
    if A is None:
        raise ValueError("A is required")
    pa, pd, pb = _whole(A, "A", _F32, dev, vec), _whole(D, "D", _F32, dev, vec), _whole(dt_bias, "dt_bias", _F32, dev, vec)
    plen, pslot = _whole(seqlens, "seqlens", _I32, dev, row), _whole(slots, "slots", _I32, dev, row)
    page = (H, P, N)
    if state_out is None:
        if slots is None:
            state_out = x.new_empty((batch, *page), dtype=_F32)
        elif init is None:
            raise ValueError("slots need a pool: init, state_out or both")
        else:
            state_out = init
    rows = _states(state_out, "state_out", dev, slots, batch, page)
    pinit = 0
    if init is not None:
        pinit = _whole(init, "init", _F32, dev, (rows, *page))
        if init is not state_out:
            _apart(init, state_out, "init", "state_out")
    if out is None:
        out = torch.empty_like(x) if x.is_contiguous() else x.new_empty(xshape)
        pout = out.data_ptr()
    else:
        pout = _whole(out, "out", io, dev, xshape)
    stream = _raw_stream(dev.index)
    ws = _scratch(dev, stream, workspace)
    nbytes = _bytes(dev.index, SSD_OP_CAUSAL_FWD, batch, L, H, P, N, G, code)
    with ws.lock:
        buf = ws.get(nbytes)
        rc = lib.ssd_causal_fwd(x.data_ptr(), dt.data_ptr(), pa, B.data_ptr(), C.data_ptr(), pd, pb, dt_min, dt_max, plen,
                                pslot, pinit, state_out.data_ptr(), pout, xs[0], xs[1], ds[0], ds[1], bs[0], bs[1],
                                cs[0], cs[1], rows, batch, L, H, P, N, G, code, path, buf.data_ptr(), buf.numel(), stream)
    _check(rc, "ssd_causal_fwd")
    return out, state_out


def ssd_causal_step(x, dt, A, B, C, D, states, slots=None, *, dt_bias=None, dt_min: float = 0.0, dt_max: float = _INF,
                    out=None, state_out=None, workspace: Workspace | None = None):
    """One token of every row (include/ssd_bidir.h: ssd_causal_step): x (batch, H,
    P), dt (batch, H), B, C (batch, G, N), D (H) or None. The states, (batch, H,
    P, N) or with slots (batch) int32 a pool of pages, advance in place unless
    state_out is given. Returns out like x."""
    got = _binding.causal_step(x, dt, A, B, C, D, states, slots, dt_bias, dt_min, dt_max, out, state_out, workspace)
    if got is not NotImplemented:
        return got
    dev, io, xshape = _lead(x, "x", 3)
    if dev.index != _device():
        with torch.cuda.device(dev):
            return ssd_causal_step(x, dt, A, B, C, D, states, slots, dt_bias=dt_bias, dt_min=dt_min, dt_max=dt_max,
                                   out=out, state_out=state_out, workspace=workspace)
    code = _DT.get(io)
    if code is None:
        raise ValueError(f"x dtype {io} not supported (float32 or bfloat16)")
    batch, H, P = xshape
    G, N = B.shape[1:] if isinstance(B, torch.Tensor) and B.dim() == 3 else (0, 0)
    bc, vec = (batch, G, N), (H,)
    xs, ds = _rows(x, "x", io, dev, xshape, 2), _rows(dt, "dt", io, dev, (batch, H), 1)
    bs, cs = _rows(B, "B", io, dev, bc, 2), _rows(C, "C", io, dev, bc, 2)
    if A is None:
        raise ValueError("A is required")
    pa, pd, pb = _whole(A, "A", _F32, dev, vec), _whole(D, "D", _F32, dev, vec), _whole(dt_bias, "dt_bias", _F32, dev, vec)
    page = (H, P, N)
    rows = _states(states, "states", dev, slots, batch, page)
    if state_out is None:
        state_out = states
    elif state_out is not states:
        _whole(state_out, "state_out", _F32, dev, (rows, *page))
        _apart(states, state_out, "states", "state_out")
    if out is None:
        out = torch.empty_like(x) if x.is_contiguous() else x.new_empty(xshape)
        pout = out.data_ptr()
    else:
        pout = _whole(out, "out", io, dev, xshape)
    stream = _raw_stream(dev.index)
    if slots is None:
        rc = lib.ssd_causal_step(x.data_ptr(), dt.data_ptr(), pa, B.data_ptr(), C.data_ptr(), pd, pb, dt_min, dt_max, 0,
                                 states.data_ptr(), state_out.data_ptr(), pout, xs[0], ds[0], bs[0], cs[0], rows, batch,
                                 H, P, N, G, code, 0, 0, stream)
    else:
        pslot = _whole(slots, "slots", _I32, dev, (batch,))
        ws = _scratch(dev, stream, workspace)
        nbytes = _bytes(dev.index, SSD_OP_CAUSAL_STEP, batch, 1, H, P, N, G, code)
        with ws.lock:
            buf = ws.get(nbytes)
            rc = lib.ssd_causal_step(x.data_ptr(), dt.data_ptr(), pa, B.data_ptr(), C.data_ptr(), pd, pb, dt_min, dt_max,
                                     pslot, states.data_ptr(), state_out.data_ptr(), pout, xs[0], ds[0], bs[0], cs[0], rows,
                                     batch, H, P, N, G, code, buf.data_ptr(), buf.numel(), stream)
    _check(rc, "ssd_causal_step")
    return out


def _pages(pool):
    """Device, layers, slots and bytes of a page of a pool (layers, slots, page...)."""
    if not isinstance(pool, torch.Tensor):
        raise TypeError("pool must be a torch.Tensor")
    dev, shape = pool.device, pool.shape
    if dev.type != "cuda":
        raise ValueError(f"pool must be a CUDA tensor (got {dev})")
    if len(shape) < 3 or not pool.is_contiguous():
        raise ValueError(f"pool must be (layers, slots, page...), contiguous (got {tuple(shape)}, strides {pool.stride()})")
    layers, nslots = shape[0], shape[1]
    if layers > _INT or nslots > _INT:
        raise ValueError(f"pool: more than {_INT} layers or slots (got {tuple(shape)})")
    return dev, layers, nslots, pool.element_size() * shape[2:].numel()


def ssd_cache_copy(pool, src, dst, *, workspace: Workspace | None = None):
    """Pages of a pool (layers, slots, ...) of any dtype, in place and in every
    layer: page dst[i] <- page src[i], or zero where src[i] is -1, in the order
    of i (include/ssd_bidir.h: ssd_cache_copy). src, dst (n) int32. Returns pool."""
    got = _binding.cache_copy(pool, src, dst, workspace)
    if got is not NotImplemented:
        return got
    dev, layers, nslots, page = _pages(pool)
    if dev.index != _device():
        with torch.cuda.device(dev):
            return ssd_cache_copy(pool, src, dst, workspace=workspace)
    if src is None or dst is None:
        raise ValueError("src and dst are required")
    n = src.shape[0] if isinstance(src, torch.Tensor) and src.dim() == 1 else 0
    ps, pd = _whole(src, "src", _I32, dev, (n,)), _whole(dst, "dst", _I32, dev, (n,))
    if n > _INT:
        raise ValueError(f"src and dst have more than {_INT} entries")
    stream = _raw_stream(dev.index)
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
    got = _binding.cache_compact(pool, table, workspace)
    if got is not NotImplemented:
        return got
    dev, layers, nslots, page = _pages(pool)
    if dev.index != _device():
        with torch.cuda.device(dev):
            return ssd_cache_compact(pool, table, workspace=workspace)
    if table is None:
        raise ValueError("table is required")
    rows = table.shape[0] if isinstance(table, torch.Tensor) and table.dim() == 1 else 0
    ptable = _whole(table, "table", _I32, dev, (rows,))
    if rows > _INT:
        raise ValueError(f"table has more than {_INT} entries")
    new, live = torch.empty_like(table), table.new_empty((1,))
    stream = _raw_stream(dev.index)
    ws = _scratch(dev, stream, workspace)
    with ws.lock:
        buf = ws.get(256)
        rc = lib.ssd_cache_compact(pool.data_ptr(), page, layers, nslots, ptable, rows, new.data_ptr(),
                                   live.data_ptr(), buf.data_ptr(), buf.numel(), stream)
    _check(rc, "ssd_cache_compact")
    return new, live
