"""Moe: a thin convenience layer over the router, dispatch and combine calls.

It allocates outputs and the workspace with PyTorch and passes raw device
addresses to libzccl, on the current CUDA stream; all work runs in the
library's kernels.  The gradients are explicit calls: ``route_backward``,
``combine_backward``, and, for a dispatch's tokens, ``combine`` without
weights.  Nothing is recorded for autograd: what a call returns does not require
a gradient, whatever its inputs do.
"""
from __future__ import annotations

import ctypes
import threading
from typing import NamedTuple, Optional

import torch

from . import (BF16, F32, OK, SCORE_SIGMOID, SCORE_SOFTMAX, Route, ZcclError, check, lib,
               zccl_dispatch_stream_bytes, zccl_dispatch_workspace_bytes)
from .codec import SEGMENT_DTYPE

_DTYPES = {torch.bfloat16: BF16, torch.float32: F32}
_SCORES = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}


class Dispatch(NamedTuple):
    """Rows in expert order and where they are."""
    rows: torch.Tensor              # [T * K, hidden]: expert 0's, expert 1's, ...; zeros after the last expert's
    pos: torch.Tensor               # int32 [T, K]: the row of each slot, -1 for none
    counts: torch.Tensor            # int32 [E]
    offsets: torch.Tensor           # int32 [E + 1]: each expert's first row; last, how many rows there are
    table: Optional[torch.Tensor]   # the 2 E segments that Codec.compress_batched reads
    streams: Optional[torch.Tensor]  # where their streams go


class Workspaces:
    """A workspace per stream, zeroed where the calls want that: calls on different
    streams must not share one.  A call that is captured into a CUDA graph gets one
    of its own, as the graph may be replayed on any stream, and so does one that
    wants more than `most` bytes.  `lock` is held from get() until the call's kernels
    are queued: they hand data over in the workspace, and a call of another host
    thread on the same stream, which gets the same one, must not come between them."""

    def __init__(self, zeroed: bool = True, most: int = 1 << 62):
        self.lock = threading.Lock()
        self._by_stream = {}
        self._new = torch.zeros if zeroed else torch.empty
        self._most = most

    def get(self, nbytes: int, stream: int, device) -> torch.Tensor:
        if nbytes > self._most or torch.cuda.is_current_stream_capturing():
            return self._new(max(nbytes, 256), dtype=torch.uint8, device=device)
        ws = self._by_stream.get(stream)
        if ws is None or ws.numel() < nbytes:
            ws = self._by_stream[stream] = self._new(max(nbytes, 256), dtype=torch.uint8, device=device)
        return ws


# The handle of the current stream, without building a Stream object where PyTorch offers it (2 us less a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def current_stream(device) -> int:
    """The handle of the current stream of `device`, which has to be the current one:
    the library launches there, and the default stream's handle is every device's."""
    if device.index != torch.cuda.current_device():
        raise ValueError(f"{device} is not the current CUDA device, on which the library's kernels run "
                         "(torch.cuda.set_device, or torch.cuda.device as a context)")
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def need(t: torch.Tensor, what: str, device, dtypes, ndim: int, rows_strided: bool = False) -> torch.Tensor:
    """Checks a tensor argument: device, type and layout (contiguous, or with
    rows_strided a matrix whose rows are contiguous)."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{what}: expected a tensor on {device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{what}: expected {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{what}: expected {ndim} dimensions, got {t.dim()}")
    if not t.is_contiguous():
        if not rows_strided:
            raise ValueError(f"{what}: expected a contiguous tensor")
        if t.shape[0] > 0 and t.shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"{what}: the values of a row have to be contiguous")
    return t


class Moe:
    """A router's configuration, its workspaces and a device status word; any
    streams and host threads may share one.

    experts, top_k: how many there are and how many a token chooses; score
    "softmax" or "sigmoid"; groups / top_groups: experts in consecutive groups of
    which a token may use the best top_groups (default: all); renormalize: divide
    a token's weights by their sum; scale: the weights' factor.  device: default
    the current one; calls refuse to run while another one is current."""

    def __init__(self, experts: int, top_k: int, *, score: str = "softmax", groups: int = 1,
                 top_groups: int | None = None, renormalize: bool = True, scale: float = 1.0, device=None):
        if score not in _SCORES:
            raise ValueError(f"score: expected one of {sorted(_SCORES)}")
        self.experts, self.top_k = int(experts), int(top_k)
        self.config = Route(self.experts, self.top_k, int(groups), int(groups if top_groups is None else top_groups),
                            _SCORES[score], 1 if renormalize else 0, float(scale))
        self._config = ctypes.addressof(self.config)
        self._lib = lib()
        # the library's own check of the configuration (no tokens: nothing is launched)
        check(self._lib.zccl_route(self._config, None, F32, 0, None, 0, None, None, None, None), "Moe")
        self.device = torch.zeros(0, device=device if device is not None else "cuda").device
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._workspaces = Workspaces()
        # the workspace for any number of tokens
        self._ws_bytes = zccl_dispatch_workspace_bytes((1 << 31) // self.top_k - 1, self.experts, self.top_k)

    # -- status ---------------------------------------------------------------
    def reset_status(self):
        self.status.zero_()

    def read_status(self) -> int:
        return int(self.status.item())

    def check_status(self, what="device"):
        st = self.read_status()
        if st != OK:
            raise ZcclError(st, what)

    # -- calls ----------------------------------------------------------------
    def _logits(self, logits):
        need(logits, "logits", self.device, _DTYPES, 2, rows_strided=True)
        tokens, experts = logits.shape
        if experts != self.experts:
            raise ValueError(f"logits: expected {self.experts} columns, got {experts}")
        return tokens, logits.stride(0), _DTYPES[logits.dtype]

    def _slots(self, t, what, dtype, tokens=None):
        need(t, what, self.device, (dtype,), 2)
        shape = t.shape
        if shape[1] != self.top_k or (tokens is not None and shape[0] != tokens):
            raise ValueError(f"{what}: expected shape [{'tokens' if tokens is None else tokens}, {self.top_k}]")
        return t

    def route(self, logits: torch.Tensor, bias: torch.Tensor | None = None):
        """(int32 [T, K] experts in order of preference, -1 for none; float32
        [T, K] weights) of logits [T, E] (BF16 or float32, rows may be strided);
        bias: float32 [E], added to the scores for the choice only."""
        tokens, stride, dtype = self._logits(logits)
        if bias is not None:
            need(bias, "bias", self.device, (torch.float32,), 1)
            if bias.shape[0] != self.experts:
                raise ValueError(f"bias: expected {self.experts} values")
        idx = torch.empty(tokens, self.top_k, dtype=torch.int32, device=self.device)
        weights = torch.empty(tokens, self.top_k, dtype=torch.float32, device=self.device)
        st = self._lib.zccl_route(self._config, logits.data_ptr(), dtype, stride,
                                  None if bias is None else bias.data_ptr(), tokens, idx.data_ptr(),
                                  weights.data_ptr(), self.status.data_ptr(), current_stream(self.device))
        check(st, "zccl_route")
        return idx, weights

    def route_backward(self, logits: torch.Tensor, idx: torch.Tensor, grad_weights: torch.Tensor) -> torch.Tensor:
        """The gradient of route's weights with respect to the logits, in the logits' type."""
        tokens, stride, dtype = self._logits(logits)
        self._slots(idx, "idx", torch.int32, tokens)
        self._slots(grad_weights, "grad_weights", torch.float32, tokens)
        grad = torch.empty(tokens, self.experts, dtype=logits.dtype, device=self.device)
        st = self._lib.zccl_route_backward(self._config, logits.data_ptr(), dtype, stride, idx.data_ptr(),
                                           grad_weights.data_ptr(), tokens, grad.data_ptr(), self.experts,
                                           current_stream(self.device))
        check(st, "zccl_route_backward")
        return grad

    def dispatch(self, x: torch.Tensor, idx: torch.Tensor, capacity: int | None = None) -> Dispatch:
        """The tokens' rows x (BF16 [T, hidden], hidden a multiple of 8, rows may be
        strided) in expert order.  With capacity (rows of an expert's static part)
        also the device-resident segment table of the batched compression, and
        room for its streams."""
        need(x, "x", self.device, (torch.bfloat16,), 2, rows_strided=True)
        tokens, hidden = x.shape
        self._slots(idx, "idx", torch.int32, tokens)
        slots = tokens * self.top_k
        rows = torch.empty(slots, hidden, dtype=torch.bfloat16, device=self.device)
        pos = torch.empty(tokens, self.top_k, dtype=torch.int32, device=self.device)
        counts = torch.empty(self.experts, dtype=torch.int32, device=self.device)
        offsets = torch.empty(self.experts + 1, dtype=torch.int32, device=self.device)
        table = streams = None
        room = 0
        if capacity is not None:
            if capacity < 0:
                raise ValueError("capacity: expected a row count")
            room = zccl_dispatch_stream_bytes(slots, hidden, self.experts)
            table = torch.empty(2 * self.experts * SEGMENT_DTYPE.itemsize, dtype=torch.uint8, device=self.device)
            streams = torch.empty(room, dtype=torch.uint8, device=self.device)
        stream = current_stream(self.device)
        with self._workspaces.lock:
            ws = self._workspaces.get(self._ws_bytes, stream, self.device)
            st = self._lib.zccl_dispatch(
                idx.data_ptr(), tokens, self.experts, self.top_k, x.data_ptr() if slots else None,
                x.stride(0) if tokens > 1 else hidden, hidden, rows.data_ptr(), pos.data_ptr(), counts.data_ptr(),
                offsets.data_ptr(), None if table is None else table.data_ptr(), capacity or 0,
                None if streams is None else streams.data_ptr(), room, ws.data_ptr(), ws.numel(), stream)
        check(st, "zccl_dispatch")
        return Dispatch(rows, pos, counts, offsets, table, streams)

    def combine(self, y: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor | None = None) -> torch.Tensor:
        """[T, hidden]: each token's rows of y (BF16 [rows, hidden]) at pos, weighted
        (without weights: added as they are) and added in fp32."""
        need(y, "y", self.device, (torch.bfloat16,), 2)
        self._slots(pos, "pos", torch.int32)
        tokens = pos.shape[0]
        if weights is not None:
            self._slots(weights, "weights", torch.float32, tokens)
        out = torch.empty(tokens, y.shape[1], dtype=torch.bfloat16, device=self.device)
        st = self._lib.zccl_combine(y.data_ptr(), y.shape[0], y.shape[1], pos.data_ptr(),
                                    None if weights is None else weights.data_ptr(), tokens, self.top_k,
                                    out.data_ptr(), current_stream(self.device))
        check(st, "zccl_combine")
        return out

    def combine_backward(self, grad: torch.Tensor, y: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor,
                         offsets: torch.Tensor):
        """(gradient of y, BF16, zero in the rows that hold no slot; float32 [T, K]
        gradient of the weights); offsets: the dispatch's."""
        need(grad, "grad", self.device, (torch.bfloat16,), 2)
        need(y, "y", self.device, (torch.bfloat16,), 2)
        need(offsets, "offsets", self.device, (torch.int32,), 1)
        tokens = grad.shape[0]
        self._slots(pos, "pos", torch.int32, tokens)
        self._slots(weights, "weights", torch.float32, tokens)
        if grad.shape[1] != y.shape[1]:
            raise ValueError("grad and y: expected the same hidden size")
        if offsets.shape[0] != self.experts + 1:
            raise ValueError(f"offsets: expected {self.experts + 1} values")
        grad_y = torch.empty_like(y)
        grad_weights = torch.empty(tokens, self.top_k, dtype=torch.float32, device=self.device)
        st = self._lib.zccl_combine_backward(grad.data_ptr(), y.data_ptr(), y.shape[0], y.shape[1], pos.data_ptr(),
                                             weights.data_ptr(), offsets.data_ptr() + 4 * self.experts, tokens,
                                             self.top_k, grad_y.data_ptr(), grad_weights.data_ptr(),
                                             current_stream(self.device))
        check(st, "zccl_combine_backward")
        return grad_y, grad_weights
