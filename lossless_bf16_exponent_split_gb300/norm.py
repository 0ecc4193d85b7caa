"""ResidualNorm and Dropout: a thin convenience layer over the calls that join a
block (a mixture of experts, a dense layer) to the residual around it.

They allocate outputs and the workspace with PyTorch and pass raw device
addresses to libzccl, on the current CUDA stream; all work runs in the
library's kernels.  The gradients are explicit calls: ``norm_backward``,
``add_backward``, and, for a dropout, ``apply`` on the gradient.  Nothing is
recorded for autograd: what a call returns does not require a gradient, whatever
its inputs do.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import BF16, F32, MAX_NORM_HIDDEN, OK, Norm, ZcclError, check, lib, zccl_residual_norm_workspace_bytes
from .moe import Workspaces, current_stream, need

_DTYPES = {torch.bfloat16: BF16, torch.float32: F32}


class ResidualGrads(NamedTuple):
    """The gradients of ResidualNorm.add's inputs; None where there is none."""
    x: torch.Tensor                       # [rows, hidden]
    y: torch.Tensor                       # [rows, hidden]
    weight: Optional[torch.Tensor]        # [hidden]
    post_weight: Optional[torch.Tensor]   # [hidden]
    gate: Optional[torch.Tensor]          # as gate


def _seed(seed):
    if not 0 <= int(seed) < 1 << 64:
        raise ValueError("seed: expected 0 .. 2^64 - 1")
    return int(seed)


def _offset(offset, device):
    """(value, address) of a dropout's offset: a number, or an int64 tensor of one value on the device."""
    if isinstance(offset, torch.Tensor):
        if offset.device != device or offset.dtype != torch.int64 or offset.numel() != 1:
            raise ValueError(f"offset: expected a number or an int64 tensor of one value on {device}")
        return 0, offset.data_ptr()
    if not 0 <= offset < 1 << 64:
        raise ValueError("offset: expected 0 .. 2^64 - 1")
    return offset, None


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stride(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


class ResidualNorm:
    """The join of a block's output with the residual, and the norm of the next
    block's input, and a device status word; any streams and host threads may share
    one.

        r = x + scale * gate * drop(b),  h = N(r; weight)
        b = N(y; post_weight) with post, else y
        N(v; w) = w * v / sqrt(mean(v^2) + eps) over a row

    hidden: values of a row; post: the block's output is normed too; scale: the
    block's factor; dropout, seed: the share of the block's output that every call
    of ``add`` drops (``Dropout``'s mask on the row and column); an evaluation has a
    handle of its own, without.  device: default the current one; calls refuse to
    run while another one is current."""

    def __init__(self, hidden: int, *, post: bool = False, eps: float = 1e-6, scale: float = 1.0, dropout: float = 0.0,
                 seed: int = 0, device=None):
        if not 0 < int(hidden) <= MAX_NORM_HIDDEN:
            raise ValueError(f"hidden: expected 1 .. {MAX_NORM_HIDDEN}")
        self.hidden, self.post = int(hidden), bool(post)
        self.config = Norm(self.hidden, 1 if post else 0, float(eps), float(scale), float(dropout), _seed(seed))
        self._config = ctypes.addressof(self.config)
        self._lib = lib()
        # the library's own check of the configuration (no rows: nothing is launched)
        check(self._lib.zccl_residual_norm(self._config, None, F32, 0, None, F32, 0, None, None, F32, None, F32, 0, 1, 0,
                                           0, None, None, None, None, None), "ResidualNorm")
        self.device = torch.zeros(0, device=device if device is not None else "cuda").device
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._status = self.status.data_ptr()
        self._workspaces = Workspaces(zeroed=False, most=64 << 20)

    # -- status ---------------------------------------------------------------
    def reset_status(self):
        self.status.zero_()

    def read_status(self) -> int:
        return int(self.status.item())

    def check_status(self, what="device"):
        st = self.read_status()
        if st != OK:
            raise ZcclError(st, what)

    # -- arguments ------------------------------------------------------------
    def _rows(self, t, what, rows=None, dtype=None):
        need(t, what, self.device, _DTYPES if dtype is None else (dtype,), 2, rows_strided=True)
        if t.shape[1] != self.hidden:
            raise ValueError(f"{what}: expected {self.hidden} columns, got {t.shape[1]}")
        if rows is not None and t.shape[0] != rows:
            raise ValueError(f"{what}: expected {rows} rows, got {t.shape[0]}")
        return t

    def _weights(self, weight, post_weight):
        """The type of the weights (which have to share one)."""
        dtype = None
        for t, what in ((weight, "weight"), (post_weight, "post_weight")):
            if t is None:
                continue
            need(t, what, self.device, _DTYPES if dtype is None else (dtype,), 1)
            if t.shape[0] != self.hidden:
                raise ValueError(f"{what}: expected {self.hidden} values, got {t.shape[0]}")
            dtype = t.dtype
        if post_weight is not None and not self.post:
            raise ValueError("post_weight: the block's output is not normed (post=False)")
        return F32 if dtype is None else _DTYPES[dtype]

    def _gate(self, gate, rows):
        """(address, type, stride, tokens of a gate row)."""
        if gate is None:
            return None, F32, 0, 1
        self._rows(gate, "gate")
        n = gate.shape[0]
        if (rows > 0 and n == 0) or (n > 0 and rows % n):
            raise ValueError(f"gate: expected a number of rows that divides {rows}, got {n}")
        return gate.data_ptr(), _DTYPES[gate.dtype], _stride(gate), max(1, rows // max(1, n))

    # -- calls ----------------------------------------------------------------
    def norm(self, x: torch.Tensor, weight: torch.Tensor | None = None, dtype: torch.dtype | None = None) -> torch.Tensor:
        """N(x; weight) of x [rows, hidden] (BF16 or float32, rows may be strided), in
        x's type or `dtype`: the first block's input."""
        self._rows(x, "x")
        wt = self._weights(weight, None)
        dtype = x.dtype if dtype is None else dtype
        if dtype not in _DTYPES:
            raise ValueError(f"dtype: expected {' or '.join(str(d) for d in _DTYPES)}, got {dtype}")
        rows = x.shape[0]
        h = torch.empty(rows, self.hidden, dtype=dtype, device=self.device)
        st = self._lib.zccl_residual_norm(self._config, x.data_ptr(), _DTYPES[x.dtype], _stride(x), None, _DTYPES[dtype], 0,
                                          _ptr(weight), None, wt, None, F32, 0, 1, rows, 0, None, None, h.data_ptr(),
                                          self._status, current_stream(self.device))
        check(st, "zccl_residual_norm")
        return h

    def norm_backward(self, grad: torch.Tensor, x: torch.Tensor, weight: torch.Tensor | None = None,
                      residual: torch.Tensor | None = None):
        """(gradient of x, in its type; gradient of the weight, in its type, or None)
        from the gradient of norm's output; residual: a gradient of x from elsewhere (of
        its type, rows may be strided), which is added."""
        self._rows(x, "x")
        rows = x.shape[0]
        self._rows(grad, "grad", rows)
        if residual is not None:
            self._rows(residual, "residual", rows, x.dtype)
        gx, _, gw, _, _ = self._backward(residual, grad, x, None, weight, None, None, 0, rows, x.dtype, grad.dtype)
        return gx, gw

    def add(self, x: torch.Tensor, y: torch.Tensor, weight: torch.Tensor | None = None, *,
            post_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None, offset=0, normed: bool = True):
        """(r, h) of the residual x and the block's output y [rows, hidden] (BF16 or
        float32 each, rows may be strided); r in x's type, h in y's, or None without
        normed.  gate [n, hidden], n dividing rows: each of its rows is that of rows / n
        consecutive tokens.  offset: the dropout's, a number or an int64 tensor of one
        value on the device, another one for each mask."""
        self._rows(x, "x")
        rows = x.shape[0]
        self._rows(y, "y", rows)
        if weight is not None and not normed:
            raise ValueError("weight: nothing is normed (normed=False)")
        wt = self._weights(weight, post_weight)
        gate_ptr, gate_type, gate_stride, span = self._gate(gate, rows)
        value, at = _offset(offset, self.device)
        r = torch.empty(rows, self.hidden, dtype=x.dtype, device=self.device)
        h = torch.empty(rows, self.hidden, dtype=y.dtype, device=self.device) if normed else None
        st = self._lib.zccl_residual_norm(self._config, x.data_ptr(), _DTYPES[x.dtype], _stride(x), y.data_ptr(),
                                          _DTYPES[y.dtype], _stride(y), _ptr(weight), _ptr(post_weight), wt, gate_ptr,
                                          gate_type, gate_stride, span, rows, value, at, r.data_ptr(), _ptr(h),
                                          self._status, current_stream(self.device))
        check(st, "zccl_residual_norm")
        return r, h

    def add_backward(self, grad_r: torch.Tensor | None, grad_h: torch.Tensor | None, r: torch.Tensor | None,
                     y: torch.Tensor, weight: torch.Tensor | None = None, *, post_weight: torch.Tensor | None = None,
                     gate: torch.Tensor | None = None, offset=0) -> ResidualGrads:
        """The gradients of add's inputs from those of r and h (either may be None, not
        both); r: the one that add returned (not needed without grad_h).  Where there
        is no grad_h the gradient of x is grad_r itself."""
        self._rows(y, "y")
        rows = y.shape[0]
        if grad_r is None and grad_h is None:
            raise ValueError("grad_r and grad_h: expected one of them at least")
        if grad_h is not None:
            self._rows(r, "r", rows)
            self._rows(grad_h, "grad_h", rows, y.dtype)
        elif weight is not None:
            raise ValueError("weight: nothing was normed (no grad_h)")
        if grad_r is not None:
            self._rows(grad_r, "grad_r", rows, None if grad_h is None else r.dtype)
        return ResidualGrads(*self._backward(grad_r, grad_h, r, y, weight, post_weight, gate, offset, rows,
                                             grad_r.dtype if grad_h is None else r.dtype, y.dtype))

    def _backward(self, grad_r, grad_h, r, y, weight, post_weight, gate, offset, rows, x_dtype, dtype):
        wt = self._weights(weight, post_weight)
        gate_ptr, gate_type, gate_stride, span = self._gate(gate, rows)
        value, at = _offset(offset, self.device)
        new = dict(device=self.device)
        gx = grad_r if grad_h is None else torch.empty(rows, self.hidden, dtype=x_dtype, **new)
        gy = None if y is None else torch.empty(rows, self.hidden, dtype=dtype, **new)
        gw, gp = (None if w is None else torch.empty(self.hidden, dtype=w.dtype, **new) for w in (weight, post_weight))
        gg = None
        if gate is not None:  # no rows: no token's gradient
            gg = (torch.empty if rows else torch.zeros)(gate.shape, dtype=gate.dtype, **new)
        stream = current_stream(self.device)
        nbytes = zccl_residual_norm_workspace_bytes(self.hidden, rows)
        with self._workspaces.lock:
            ws = self._workspaces.get(nbytes, stream, self.device)
            st = self._lib.zccl_residual_norm_backward(
                self._config, _ptr(grad_r), 0 if grad_r is None else _stride(grad_r), _ptr(grad_h),
                0 if grad_h is None else _stride(grad_h), None if grad_h is None else r.data_ptr(), _DTYPES[x_dtype],
                0 if grad_h is None else _stride(r), _ptr(y), _DTYPES[dtype], 0 if y is None else _stride(y), _ptr(weight),
                _ptr(post_weight), wt, gate_ptr, gate_type, gate_stride, span, rows, value, at,
                None if grad_h is None else gx.data_ptr(), _ptr(gy), _ptr(gw), _ptr(gp), _ptr(gg), ws.data_ptr(),
                ws.numel(), self._status, stream)
        check(st, "zccl_residual_norm_backward")
        return gx, gy, gw, gp, gg


class Dropout:
    """Dropout whose mask is a function of seed, offset, row and column and is never
    stored: the gradient is the same call on the output's gradient.  p: the share
    that is dropped, rounded to a multiple of 2^-16; what is kept is divided by
    1 - p.  device: default the current one; calls refuse to run while another one
    is current."""

    def __init__(self, p: float, *, seed: int = 0, device=None):
        if not 0.0 <= p <= 1.0:
            raise ValueError("p: expected 0 .. 1")
        self.p, self.seed = float(p), _seed(seed)
        self._lib = lib()
        self.device = torch.zeros(0, device=device if device is not None else "cuda").device

    def apply(self, x: torch.Tensor, offset=0, out: torch.Tensor | None = None) -> torch.Tensor:
        """x [rows, cols] (BF16 or float32, rows may be strided) with its dropped
        elements zero; offset: a number or an int64 tensor of one value on the device,
        another one for each mask.  out: where the result goes (x itself, for one)."""
        need(x, "x", self.device, _DTYPES, 2, rows_strided=True)
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=self.device)
        else:
            need(out, "out", self.device, (x.dtype,), 2)
            if out.shape != x.shape:
                raise ValueError(f"out: expected shape {tuple(x.shape)}")
        value, at = _offset(offset, self.device)
        st = self._lib.zccl_dropout(x.data_ptr(), _DTYPES[x.dtype], _stride(x), x.shape[0], x.shape[1], self.p, self.seed,
                                    value, at, out.data_ptr(), current_stream(self.device))
        check(st, "zccl_dropout")
        return out
