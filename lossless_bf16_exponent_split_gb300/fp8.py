"""BlockFp8: a thin convenience layer over the block-scaled e4m3 layers.

Outputs and workspaces come from PyTorch, raw device addresses go to libzccl on
the current CUDA stream; quantisation and products run in the library's kernels.
The gradients are an explicit call, ``linear_backward``; nothing is recorded for
autograd: what a call returns does not require a gradient, whatever its inputs do.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import (BF16, F32, OK, ZcclError, check, lib, zccl_fp8_linear_workspace_bytes, zccl_fp8_weight_bytes)
from .moe import Workspaces, current_stream, need

_DTYPES = {torch.bfloat16: BF16, torch.float32: F32}
BLOCK = 128


class Fp8Weight(NamedTuple):
    """A packed weight of `groups` matrices [n, k]."""
    groups: int
    n: int
    k: int
    packed: torch.Tensor                # what linear reads
    packed_t: Optional[torch.Tensor]    # what the gradient of the input reads


class BlockFp8:
    """A device status word, workspaces and the calls of the block-scaled e4m3 layers;
    any streams and host threads may share one.  device: default the current one;
    calls refuse to run while another one is current."""

    def __init__(self, device=None):
        self._lib = lib()
        self.device = torch.zeros(0, device=device if device is not None else "cuda").device
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        # a call's workspace costs 1.5 us to allocate: a serving step's is kept, a large one is not
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

    # -- weights --------------------------------------------------------------
    def _buffers(self, groups, n, k, backward):
        packed = torch.empty(zccl_fp8_weight_bytes(groups, n, k), dtype=torch.uint8, device=self.device)
        packed_t = torch.empty(zccl_fp8_weight_bytes(groups, k, n), dtype=torch.uint8, device=self.device) if backward else None
        return packed, packed_t

    def quantize_weight(self, w: torch.Tensor, backward: bool = False) -> Fp8Weight:
        """Packs w [groups, n, k] (or [n, k]; BF16 or float32); with backward also what
        linear_backward reads."""
        w = w.unsqueeze(0) if torch.is_tensor(w) and w.dim() == 2 else w
        need(w, "w", self.device, _DTYPES, 3)
        packed, packed_t = self._buffers(*w.shape, backward)
        st = self._lib.zccl_fp8_weight_quantize(w.data_ptr(), _DTYPES[w.dtype], *w.shape, packed.data_ptr(),
                                                None if packed_t is None else packed_t.data_ptr(),
                                                current_stream(self.device))
        check(st, "zccl_fp8_weight_quantize")
        return Fp8Weight(*w.shape, packed, packed_t)

    def weight(self, codes: torch.Tensor, scale: torch.Tensor, backward: bool = False) -> Fp8Weight:
        """Packs a weight held as e4m3 codes [groups, n, k] and float32 scales of its
        128 x 128 blocks [groups, n/128, k/128] (rounded up), e.g. a checkpoint's."""
        need(codes, "codes", self.device, (torch.float8_e4m3fn,), 3)
        need(scale, "scale", self.device, (torch.float32,), 3)
        groups, n, k = codes.shape
        if tuple(scale.shape) != (groups, -(-n // BLOCK), -(-k // BLOCK)):
            raise ValueError(f"scale: expected shape {(groups, -(-n // BLOCK), -(-k // BLOCK))}")
        packed, packed_t = self._buffers(groups, n, k, backward)
        st = self._lib.zccl_fp8_weight_pack(codes.data_ptr(), scale.data_ptr(), groups, n, k, packed.data_ptr(),
                                            None if packed_t is None else packed_t.data_ptr(),
                                            current_stream(self.device))
        check(st, "zccl_fp8_weight_pack")
        return Fp8Weight(groups, n, k, packed, packed_t)

    # -- products -------------------------------------------------------------
    def _offsets(self, offsets, weight):
        if offsets is None:
            if weight.groups != 1:
                raise ValueError("offsets: needed for more than one group")
            return None
        need(offsets, "offsets", self.device, (torch.int32,), 1)
        if offsets.shape[0] != weight.groups + 1:
            raise ValueError(f"offsets: expected {weight.groups + 1} values")
        return offsets.data_ptr()

    def _rows(self, t, what, cols):
        need(t, what, self.device, _DTYPES, 2, rows_strided=True)
        if t.shape[1] != cols:
            raise ValueError(f"{what}: expected {cols} columns, got {t.shape[1]}")
        return t.data_ptr(), (t.stride(0) if t.shape[0] > 1 else cols)

    def linear(self, x: torch.Tensor, weight: Fp8Weight, offsets: torch.Tensor | None = None,
               out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """[rows, n]: each row of x [rows, k] (BF16 or float32, rows may be strided)
        times its group's weight; offsets: int32 [groups + 1], each group's first row
        (a dispatch's).  Rows after the last group's give zeros."""
        ptr, stride = self._rows(x, "x", weight.k)
        off = self._offsets(offsets, weight)
        rows = x.shape[0]
        out = torch.empty(rows, weight.n, dtype=out_dtype, device=self.device)
        stream = current_stream(self.device)
        nbytes = zccl_fp8_linear_workspace_bytes(rows, weight.k, weight.n, weight.groups, False)
        with self._workspaces.lock:
            ws = self._workspaces.get(nbytes, stream, self.device)
            st = self._lib.zccl_fp8_linear(ptr, _DTYPES[x.dtype], stride, rows, weight.k, weight.packed.data_ptr(), weight.n,
                                           weight.groups, off, out.data_ptr(), _out_type(out_dtype), ws.data_ptr(),
                                           ws.numel(), self.status.data_ptr(), stream)
        check(st, "zccl_fp8_linear")
        return out

    def linear_backward(self, grad: torch.Tensor, x: torch.Tensor, weight: Fp8Weight,
                        offsets: torch.Tensor | None = None, *, input_grad: bool = True, weight_grad: bool = True,
                        out_dtype: torch.dtype = torch.bfloat16):
        """(gradient of x [rows, k], gradient of the weight [groups, n, k]) from the
        gradient [rows, n] of linear's output; None for the one not asked for."""
        gptr, gstride = self._rows(grad, "grad", weight.n)
        xptr, xstride = self._rows(x, "x", weight.k)
        off = self._offsets(offsets, weight)
        rows = grad.shape[0]
        if x.shape[0] != rows or x.dtype != grad.dtype:
            raise ValueError("x and grad: expected as many rows, of the same type")
        if input_grad and weight.packed_t is None:
            raise ValueError("weight: packed without backward=True")
        dx = torch.empty(rows, weight.k, dtype=out_dtype, device=self.device) if input_grad else None
        dw = torch.empty(weight.groups, weight.n, weight.k, dtype=out_dtype, device=self.device) if weight_grad else None
        stream = current_stream(self.device)
        nbytes = zccl_fp8_linear_workspace_bytes(rows, weight.k, weight.n, weight.groups, True)
        with self._workspaces.lock:
            ws = self._workspaces.get(nbytes, stream, self.device)
            st = self._lib.zccl_fp8_linear_backward(
                gptr, xptr, _DTYPES[grad.dtype], gstride, xstride, rows, weight.k,
                None if weight.packed_t is None else weight.packed_t.data_ptr(), weight.n, weight.groups, off,
                None if dx is None else dx.data_ptr(), None if dw is None else dw.data_ptr(), _out_type(out_dtype),
                ws.data_ptr(), ws.numel(), self.status.data_ptr(), stream)
        check(st, "zccl_fp8_linear_backward")
        return dx, dw


def _out_type(dtype):
    if dtype not in _DTYPES:
        raise ValueError(f"out_dtype: expected {' or '.join(str(d) for d in _DTYPES)}, got {dtype}")
    return _DTYPES[dtype]
