"""Binding of the compressed source cache (see include/attnres.h).

Rows of sources are held in 8 or 4 bits per channel: attnres_cache_write
quantises them, attnres_cache_load reads them back, attnres_cached_fwd and
attnres_cached_bwd are the read and its gradient over cached sources, and
attnres_cached is the autograd operator.  Records are uint8 tensors
[..., attnres_cache_row_bytes(D, bits)]; S of them (packed [S, ..., bytes], or
a list) are the sources of a read.  As in ops.py, only pointers and sizes are
marshalled here and CPU tensors are rejected.  A call runs on the current
stream of its tensors' device, or on `stream` as if that one were current.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache
from typing import Optional, Sequence, Union

import torch

from . import _lib
from .ops import EPS_DEFAULT, _as_rows, _check_out, _check_vec, _out_rows

Records = Union[torch.Tensor, Sequence[torch.Tensor]]


@lru_cache(maxsize=None)
def attnres_cache_row_bytes(D: int, bits: int) -> int:
    """Bytes of one token's record (a multiple of 16)."""
    n = int(_lib.load().attnres_cache_row_bytes(int(D), int(bits)))
    if n == 0:
        raise ValueError(f"the cache takes bits 8 or 4 and D a multiple of 8 in 8..{_lib.MAX_D}")
    return n


def _call(name: str, device, *args) -> None:
    """The library's function `name` with `args` and the current stream of the
    tensors' device, that device current."""
    f = getattr(_lib.load(), name)
    index = device.index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if index == torch.cuda.current_device():
        rc = f(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = f(*args, stream)
    if rc:
        _lib.check(rc, name)


def _on(stream, rows: Records):
    """Makes `stream` current: what a call allocates and the copies it makes of
    inputs that it cannot address belong to the stream that it runs on."""
    if not isinstance(rows, torch.Tensor) and not len(rows):
        raise ValueError("need at least one cached source")
    t = rows if isinstance(rows, torch.Tensor) else rows[0]
    if not t.is_cuda:
        raise TypeError("needs CUDA tensors")
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=t.device) if stream else \
            torch.cuda.default_stream(t.device)
    if stream.device != t.device:
        raise ValueError("stream must be on the tensors' device")
    return torch.cuda.stream(stream)


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _aligned(t: torch.Tensor) -> torch.Tensor:
    """Contiguous and on a 16-byte boundary (a copy where it is not)."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _bf16_rows(t: torch.Tensor, name: str):
    """(address, tokens, elements between rows, what keeps the rows alive); a
    copy is made where the rows cannot be addressed."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA bf16 tensor")
    D = t.shape[-1]
    if t.is_contiguous():
        r, n, ld = t, t.numel() // D if D else 0, D
    else:
        r = _as_rows(t, D)
        n, ld = r.shape[0], r.stride(0) if r.shape[0] > 1 else D
    if r.data_ptr() % 16 or ld % 8:
        r, ld = _aligned(r), D
    return r.data_ptr(), n, ld, r


def _record_rows(t: torch.Tensor, size: int, writable: bool = False):
    """(address, tokens, bytes between records, what keeps them alive)."""
    if t.dtype != torch.uint8 or not t.is_cuda:
        raise TypeError("records must be CUDA uint8 tensors")
    if t.dim() < 1 or t.shape[-1] != size:
        raise ValueError(f"records must be [..., {size}] for this D and bits")
    n = t.numel() // size
    if t.is_contiguous() and t.data_ptr() % 16 == 0:
        return t.data_ptr(), n, size, t
    try:
        r = t.view(-1, size) if n else t.reshape(0, size)
    except RuntimeError as e:
        if writable:
            raise ValueError("out: records must be addressable as [N, bytes]") from e
        r = t.contiguous().view(-1, size)
    ld = r.stride(0) if n > 1 else size
    if (n and r.stride(1) != 1) or r.data_ptr() % 16 or ld % 16 or ld < size:
        if writable:
            raise ValueError("out: records must be dense, 16-byte aligned and not overlap")
        r, ld = _aligned(r), size
    return r.data_ptr(), n, ld, r


class _Sources:
    """The records of a read's sources: addresses, tokens, leading shape."""

    __slots__ = ("addrs", "keep", "N", "ld", "lead", "device", "packed")

    def __init__(self, rows: Records, size: int):
        if isinstance(rows, torch.Tensor):
            if rows.dim() < 2 or rows.shape[0] < 1:
                raise ValueError("packed records must be [S, ..., bytes] with S >= 1")
            S = rows.shape[0]
            self.packed, self.lead, self.device = True, rows.shape[1:-1], rows.device
            if rows.is_contiguous() and rows.data_ptr() % 16 == 0:
                base, total, self.ld, self.keep = _record_rows(rows, size)
                self.N = total // S
                step = self.N * size
            else:
                base, self.N, self.ld, self.keep = _record_rows(rows[0], size)
                step = rows.stride(0)
                if base != rows.data_ptr() or step % 16:   # the first source could not be addressed in place
                    self.keep = _aligned(rows)
                    base, self.ld, step = self.keep.data_ptr(), size, self.N * size
                else:
                    self.keep = rows
            self.addrs = [base + s * step for s in range(S)]
            return
        rows = list(rows)
        if not rows:
            raise ValueError("need at least one cached source")
        self.packed, self.lead, self.device = False, rows[0].shape[:-1], rows[0].device
        for r in rows:
            if r.shape[:-1] != self.lead:
                raise ValueError("all sources must have the same shape")
            if r.device != self.device:
                raise ValueError("all sources must be on one device")
        found = [_record_rows(r, size) for r in rows]
        if len({ld for _, _, ld, _ in found}) > 1:
            found = [_record_rows(_aligned(r), size) for r in rows]
        self.addrs, self.keep = [f[0] for f in found], [f[3] for f in found]
        self.N, self.ld = found[0][1], found[0][2]


def _params(src: _Sources, R: int, D: int, bits: int, live, key_offset, eps, scale, out_norm: bool):
    S = len(src.addrs)
    if S + (live is not None) > _lib.MAX_S:
        raise ValueError(f"at most {_lib.MAX_S} sources")
    p = _lib.AttnresCachedParams()
    p.S, p.D, p.R, p.N, p.bits = S, D, R, src.N, bits
    p.key_offset = D - R if key_offset is None else int(key_offset)
    p.eps, p.scale, p.out_norm = float(eps), float(scale), int(out_norm)
    p.row_ld = src.ld
    p.rows[:S] = src.addrs
    keep = None
    if live is not None:
        if tuple(live.shape) != (*src.lead, D):
            raise ValueError("live must have the cached sources' leading shape and D channels")
        if live.device != src.device:
            raise ValueError("live must be on the records' device")
        p.live, _, p.live_ld, keep = _bf16_rows(live, "live")
    return p, keep


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on the records' device")


def attnres_cache_write(values: torch.Tensor, *, bits: int = 8, key_rank: Optional[int] = None,
                        key_offset: Optional[int] = None, out: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """Quantise [..., D] bf16 rows into records, uint8 [..., bytes], for reads
    whose key is the key_rank channels (default D) from key_offset on (default
    the last ones).  ``out`` may be part of a larger cache, such as one
    source's tokens from t on: ``cache[s, t:t + n]``."""
    if torch.compiler.is_compiling() and out is None and stream is None:
        from .custom_ops import cache_write
        D = values.shape[-1]
        R = D if key_rank is None else key_rank
        return cache_write(values, bits, R, D - R if key_offset is None else key_offset)
    if stream is not None:
        with _on(stream, values):
            return attnres_cache_write(values, bits=bits, key_rank=key_rank, key_offset=key_offset, out=out)
    x, N, ld, keep = _bf16_rows(values, "values")
    D, dev = values.shape[-1], values.device
    size = attnres_cache_row_bytes(D, bits)
    R = D if key_rank is None else int(key_rank)
    shape = (*values.shape[:-1], size)
    given = out is not None
    if not given:
        out = torch.empty(shape, dtype=torch.uint8, device=dev)
    elif out.shape != shape:
        raise ValueError(f"out must be uint8 {list(shape)}")
    _same_device(dev, out=out)
    rows, _, row_ld, _ = _record_rows(out, size, writable=True)
    _call("attnres_cache_write", dev, x, ld, N, D, int(bits), R,
          D - R if key_offset is None else int(key_offset), rows, row_ld)
    if given and not out.is_inference():    # a read whose backward still needs the old records finds out
        torch.autograd.graph.increment_version(out)
    return out


def attnres_cache_load(rows: torch.Tensor, D: int, *, bits: int = 8, out: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """Read records back: bf16 [..., D], exactly the values that reads of the cache use."""
    if torch.compiler.is_compiling() and out is None and stream is None:
        from .custom_ops import cache_load
        return cache_load(rows, D, bits)
    if stream is not None:
        with _on(stream, rows):
            return attnres_cache_load(rows, D, bits=bits, out=out)
    size = attnres_cache_row_bytes(D, bits)
    src, N, row_ld, keep = _record_rows(rows, size)
    shape, dev = (*rows.shape[:-1], D), rows.device
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        dst, ld = out.data_ptr(), D
    else:
        if out.shape != shape:
            raise ValueError(f"out must be bf16 {list(shape)}")
        _same_device(dev, out=out)
        r = _out_rows(out, N, D, "out")
        dst, ld = r.data_ptr(), r.stride(0) if N > 1 else D
        if dst % 16 or ld % 8 or ld < D:
            raise ValueError("out: rows must start on 16-byte boundaries and not overlap")
    _call("attnres_cache_load", dev, src, row_ld, N, D, int(bits), dst, ld)
    return out


def attnres_cached_fwd(rows: Records, q: torch.Tensor, D: int, *, bits: int = 8, live: Optional[torch.Tensor] = None,
                       w_o: Optional[torch.Tensor] = None, eps: float = EPS_DEFAULT, scale: float = 1.0,
                       key_offset: Optional[int] = None, stream=None, out: Optional[dict] = None) -> dict:
    """The read over cached sources and, last, an optional bf16 source `live`
    [..., D].  Returns y [..., D] and the statistics alpha/rstd/logit
    [N, sources] and, with w_o, o_rstd [N].  `out` may supply tensors."""
    if stream is not None:
        with _on(stream, rows):
            return attnres_cached_fwd(rows, q, D, bits=bits, live=live, w_o=w_o, eps=eps, scale=scale,
                                      key_offset=key_offset, out=out)
    D = int(D)
    src = _Sources(rows, attnres_cache_row_bytes(D, bits))
    dev, N, S = src.device, src.N, len(src.addrs) + (live is not None)
    R = q.numel()
    q = _check_vec(q, R, "q")
    w_o = None if w_o is None else _aligned(_check_vec(w_o, D, "w_o"))
    _same_device(dev, q=q, w_o=w_o)
    p, keep = _params(src, R, D, int(bits), live, key_offset, eps, scale, w_o is not None)
    f32 = torch.float32
    o_rstd = None
    if out:
        y, alpha, rstd, logit = (out.get(k) for k in ("y", "alpha", "rstd", "logit"))
        _check_out(y, N * D, torch.bfloat16, "y", dev)
        for name in ("alpha", "rstd", "logit"):
            _check_out(out.get(name), N * S, f32, name, dev)
        if w_o is not None:
            o_rstd = out.get("o_rstd")
            _check_out(o_rstd, N, f32, "o_rstd", dev)
    else:
        y = alpha = rstd = logit = None
    shape = (*src.lead, D)
    y = torch.empty(shape, dtype=torch.bfloat16, device=dev) if y is None else y.view(shape)
    alpha = torch.empty((N, S), dtype=f32, device=dev) if alpha is None else alpha
    rstd = torch.empty((N, S), dtype=f32, device=dev) if rstd is None else rstd
    logit = torch.empty((N, S), dtype=f32, device=dev) if logit is None else logit
    if w_o is not None and o_rstd is None:
        o_rstd = torch.empty((N,), dtype=f32, device=dev)
    _call("attnres_cached_fwd", dev, ctypes.byref(p), q.data_ptr(), _addr(w_o), y.data_ptr(), alpha.data_ptr(),
          rstd.data_ptr(), logit.data_ptr(), _addr(o_rstd))
    return {"y": y, "alpha": alpha, "rstd": rstd, "logit": logit, "o_rstd": o_rstd}


def _workspace_bytes(params: _lib.AttnresCachedParams, device) -> int:
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return int(_lib.load().attnres_cached_bwd_workspace_bytes(ctypes.byref(params)))
    return int(_lib.load().attnres_cached_bwd_workspace_bytes(ctypes.byref(params)))


def attnres_cached_bwd(rows: Records, q: torch.Tensor, dy: torch.Tensor, saved: dict, D: int, *, bits: int = 8,
                       live: Optional[torch.Tensor] = None, w_o: Optional[torch.Tensor] = None,
                       eps: float = EPS_DEFAULT, scale: float = 1.0, key_offset: Optional[int] = None, stream=None,
                       need_dvalues: bool = True, need_dlive: bool = True, dvalues: Optional[Records] = None,
                       workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradient of attnres_cached_fwd; `saved` is its result.  Returns dvalues
    (packed [S, ..., D] if the records were packed, else a list; the gradient
    of the values that the codes stand for, which passed straight through is
    that of the rows written; None without need_dvalues), d_live, and dq/dw_o
    in bf16 and fp32.  `dvalues` and `workspace` may be given."""
    if stream is not None:
        with _on(stream, rows):
            return attnres_cached_bwd(rows, q, dy, saved, D, bits=bits, live=live, w_o=w_o, eps=eps, scale=scale,
                                      key_offset=key_offset, need_dvalues=need_dvalues, need_dlive=need_dlive,
                                      dvalues=dvalues, workspace=workspace)
    D = int(D)
    src = _Sources(rows, attnres_cache_row_bytes(D, bits))
    dev, N, S = src.device, src.N, len(src.addrs)
    R = q.numel()
    q = _check_vec(q, R, "q")
    w_o = None if w_o is None else _aligned(_check_vec(w_o, D, "w_o"))
    if dy.dtype != torch.bfloat16 or not dy.is_cuda or dy.numel() != N * D:
        raise TypeError("dy must be a CUDA bf16 tensor shaped like the output")
    dy = _aligned(dy)
    _same_device(dev, q=q, w_o=w_o, dy=dy, workspace=workspace)
    p, keep = _params(src, R, D, int(bits), live, key_offset, eps, scale, w_o is not None)
    total = S + (live is not None)
    for name in ("alpha", "rstd", "logit"):
        _check_out(saved[name], N * total, torch.float32, name, dev)
    if w_o is not None:
        _check_out(saved["o_rstd"], N, torch.float32, "o_rstd", dev)
    shape = (*src.lead, D)
    dptrs, dld = None, D
    if not need_dvalues:
        dvalues = None
    else:
        if dvalues is None:
            if src.packed:
                dvalues = torch.empty((S, *shape), dtype=torch.bfloat16, device=dev)
                base, step = dvalues.data_ptr(), N * D * 2
                addrs = [base + s * step for s in range(S)]
            else:
                dvalues = [torch.empty(shape, dtype=torch.bfloat16, device=dev) for _ in range(S)]
                addrs = [d.data_ptr() for d in dvalues]
        else:
            given = list(dvalues)
            if len(given) != S:
                raise ValueError("dvalues: one gradient per cached source")
            given = [_out_rows(d, N, D, "dvalues") for d in given]
            for d in given:
                _same_device(dev, dvalues=d)
            dld = given[0].stride(0) if N > 1 else D
            if N > 1 and any(d.stride(0) != dld for d in given):
                raise ValueError("dvalues: every source's gradient rows need the same row stride")
            addrs = [d.data_ptr() for d in given]
        dptrs = (ctypes.c_void_p * S)(*addrs)
    d_live = torch.empty(shape, dtype=torch.bfloat16, device=dev) if live is not None and need_dlive else None
    dq = torch.empty((R,), dtype=torch.bfloat16, device=dev)
    dq32 = torch.empty((R,), dtype=torch.float32, device=dev)
    dw = dw32 = None
    if w_o is not None:
        dw = torch.empty((D,), dtype=torch.bfloat16, device=dev)
        dw32 = torch.empty((D,), dtype=torch.float32, device=dev)
    need = _workspace_bytes(p, dev)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty((max(need, 16),), dtype=torch.uint8, device=dev)
    _call("attnres_cached_bwd", dev, ctypes.byref(p), q.data_ptr(), _addr(w_o), dy.data_ptr(),
          saved["alpha"].data_ptr(), saved["rstd"].data_ptr(), saved["logit"].data_ptr(), _addr(saved.get("o_rstd")),
          dptrs, dld, _addr(d_live), D, dq.data_ptr(), dq32.data_ptr(), _addr(dw), _addr(dw32), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return {"dvalues": dvalues, "d_live": d_live, "dq": dq, "dq_f32": dq32, "dw_o": dw, "dw_o_f32": dw32}


def attnres_cached(rows: Records, query: torch.Tensor, D: int, *, bits: int = 8,
                   values: Optional[Records] = None, live: Optional[torch.Tensor] = None, eps: float = EPS_DEFAULT,
                   scale: float = 1.0, out_norm_weight: Optional[torch.Tensor] = None,
                   key_offset: Optional[int] = None) -> torch.Tensor:
    """AttnRes read over cached sources (see attnres): returns [..., D] bf16.

    rows: records written by attnres_cache_write for this key slice, packed
    [S, ..., bytes] or a list of [..., bytes].  live: an optional bf16 source
    read last.  values: the tensors the records were written from (packed or a
    list, as the rows); they are not read or kept, but receive the gradient of
    the cached values, passed straight through the rounding.  Differentiable
    in values, live, query and out_norm_weight; a registered torch operator.
    The records are kept for the backward: until it has run no source read may
    be written again.  Autograd notices a write into a source's own tensor;
    sources that share one tensor (packed) count as written together, so give
    each a tensor of its own where later ones are written before the backward.
    To capture the gradient in a CUDA graph use torch.autograd.grad, with no
    eager graph of the same leaves alive."""
    from .custom_ops import attnres_cached_op
    return attnres_cached_op(rows, query, D, bits=bits, values=values, live=live, eps=eps, scale=scale,
                             out_norm_weight=out_norm_weight, key_offset=key_offset)
