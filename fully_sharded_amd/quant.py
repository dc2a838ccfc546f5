"""8-bit codes: the binding of fsdp_quantize_rows and of the all-gather in 8
bits, fsdp_quant_*, fsdp_gather_quantize and fsdp_dequantize (see
include/fsdp_mi355x.h).

    qu = Quant(plan)                                   # which parameters travel in 8 bits
    codes = [qu.code_buffer() for _ in range(plan.R)]  # what every rank receives
    scales = [qu.scale_buffer() for _ in range(plan.R)]
    rest = [qu.rest_buffer() for _ in range(plan.R)]
    fsdp_gather_quantize(qu, shards, codes, scales, rest)
    Wq, sw = qu.codes(codes[r])[0], qu.scales(scales[r])[0]
    fsdp_quantize_rows(x, xq, sx)                      # the rank's activations
    fsdp_grouped_matmul_i8("nt", xq, sx, Wq, sw, y)    # y = x W^T
    fsdp_quantize_rows(dy, dq, sd, channel=sw)         # the weights' scales taken in
    fsdp_grouped_matmul_i8("nn", dq, sd, Wq, None, dx) # dx = dy W
    fsdp_dequantize(qu, codes, scales, rest, units)    # or units of bf16 again

Every call runs on the GPU that holds its tensors, which has to be the current
one, and on the current stream unless another is given; tensors of a call on
another stream have to live until it is done there.  The bind_* forms check the
tensors and marshal the pointers once, for loops.
"""

from __future__ import annotations

import ctypes
import sys

import torch

from . import binding as _b
from .binding import Plan, _check, _dev, _dtype_code, _ptr_array, _stream, lib
from .muon import _bound
from .products import _codes, _matrix, _offsets, _pitch, _row_stride, _scales


class Quant:
    """The parameters of `plan` that travel in 8 bits (their indices; by
    default every parameter of two dimensions or more), with a scale for every
    row along their last dimension."""

    def __init__(self, plan: Plan, params=None):
        if params is None:
            params = [p for p, s in enumerate(plan.shapes) if len(s) >= 2]
        params = [int(p) for p in params]
        arr = (ctypes.c_int32 * max(1, len(params)))(*params)
        h = ctypes.c_void_p()
        _check("fsdp_quant_plan", lib().fsdp_quant_plan(plan.handle, len(params), arr,
                                                        ctypes.byref(h)))
        self._h = h
        self.plan = plan
        self.params = params
        out = (ctypes.c_int64 * 3)()
        _check("fsdp_quant_sizes", lib().fsdp_quant_sizes(h, out))
        self.code_bytes, self.n_scales, self.rest_numel = out
        self._at = []
        for p in range(plan.n_params):
            at = (ctypes.c_int64 * 5)()
            _check("fsdp_quant_param", lib().fsdp_quant_param(h, p, at))
            self._at.append(tuple(at))

    @property
    def handle(self):
        return self._h

    def __del__(self):
        # at interpreter exit the HIP runtime may already be gone: leak then
        h = getattr(self, "_h", None)
        if h is not None and _b._lib is not None and not sys.is_finalizing():
            _b._lib.fsdp_quant_destroy(h)
            self._h = None

    def prepare(self, stream=None):
        """Upload the work table to the current device now."""
        _check("fsdp_quant_prepare", lib().fsdp_quant_prepare(self._h, _stream(stream)))

    def code_buffer(self, device="cuda"):
        """A receiver's codes, uninitialised."""
        return torch.empty(self.code_bytes, dtype=torch.int8, device=device)

    def scale_buffer(self, device="cuda"):
        """A receiver's scales, uninitialised."""
        return torch.empty(self.n_scales, dtype=torch.float32, device=device)

    def rest_buffer(self, dtype=torch.bfloat16, device="cuda"):
        """A receiver's other parameters, uninitialised."""
        return torch.empty(self.rest_numel, dtype=dtype, device=device)

    def codes(self, buf):
        """The chosen parameters' codes in a receiver's buffer, in the order of
        `params`: views of their shapes, rows at multiples of 16 bytes."""
        out = []
        for p in self.params:
            to, rows, cols, pitch, _ = self._at[p]
            strides, step = [1], pitch
            for d in reversed(self.plan.shapes[p][:-1]):
                strides.append(step)
                step *= d
            out.append(buf.as_strided(self.plan.shapes[p], strides[::-1],
                                      buf.storage_offset() + to))
        return out

    def scales(self, buf):
        """Their scales, one per row: views of their shapes without the last
        dimension."""
        return [buf[self._at[p][4]:self._at[p][4] + self._at[p][1]].view(self.plan.shapes[p][:-1])
                for p in self.params]

    def rest(self, buf):
        """The other parameters, in the plan's order: views of their shapes."""
        return [buf[at[1]:at[1] + at[2]].view(s)
                for at, s in zip(self._at, self.plan.shapes) if at[0] < 0]


def fsdp_quant_plan(plan: Plan, params=None) -> Quant:
    return Quant(plan, params)


def _receivers(qu, what, buffers, numel, dtype=None):
    """R tensors of numel elements (None: skipped), and their dtype."""
    buffers = list(buffers)
    if len(buffers) != qu.plan.R:
        raise ValueError(f"need R buffers of {what}")
    for t in buffers:
        if t is None:
            continue
        if t.numel() != numel:
            raise ValueError(f"{what} must have {numel} elements")
        if dtype is None:
            dtype = t.dtype
        if numel and t.dtype != dtype:
            raise ValueError(f"{what} must be {dtype}")
    return buffers, dtype


def bind_gather_quantize(qu: Quant, shards, codes, scales, rest):
    """fsdp_gather_quantize with cached arguments; call as f(stream=None)."""
    if shards.numel() != qu.plan.R * qu.plan.S:
        raise ValueError("shards must have R*S elements")
    dt = _dtype_code(shards)
    codes, _ = _receivers(qu, "codes", codes, qu.code_bytes, torch.int8)
    scales, _ = _receivers(qu, "scales", scales, qu.n_scales, torch.float32)
    rest, _ = _receivers(qu, "rest", rest, qu.rest_numel, shards.dtype)
    args = (qu.handle, ctypes.c_void_p(_dev(shards, "shards")), dt, _ptr_array(codes, "codes"),
            _ptr_array(scales, "scales"), _ptr_array(rest, "rest"))
    tensors = [t for t in (shards, *codes, *scales, *rest) if t is not None]
    return _bound("fsdp_gather_quantize", args, (qu, tensors), tensors)


def fsdp_gather_quantize(qu: Quant, shards, codes, scales, rest, stream=None):
    """shards [R, S] -> every receiver's codes, scales and rest (lists of R
    tensors; where codes has None, that receiver is skipped)."""
    bind_gather_quantize(qu, shards, codes, scales, rest)(stream)


def bind_dequantize(qu: Quant, codes, scales, rest, full_out):
    """fsdp_dequantize with cached arguments; call as f(stream=None)."""
    codes, _ = _receivers(qu, "codes", codes, qu.code_bytes, torch.int8)
    scales, _ = _receivers(qu, "scales", scales, qu.n_scales, torch.float32)
    rest, rest_type = _receivers(qu, "rest", rest, qu.rest_numel)
    full_out, out_type = _receivers(qu, "full_out", full_out, qu.plan.T)
    if out_type is None:
        raise ValueError("need a unit to write")

    def code(dtype):
        return _b.BF16 if dtype is None else _dtype_code(torch.empty(0, dtype=dtype))
    args = (qu.handle, _ptr_array(codes, "codes"), _ptr_array(scales, "scales"),
            _ptr_array(rest, "rest"), code(rest_type), _ptr_array(full_out, "full_out"),
            code(out_type))
    tensors = [t for t in (*full_out, *codes, *scales, *rest) if t is not None]
    return _bound("fsdp_dequantize", args, (qu, tensors), tensors)


def fsdp_dequantize(qu: Quant, codes, scales, rest, full_out, stream=None):
    """Every receiver's buffers -> its unit [T], bf16 or fp32 (lists of R
    tensors; where full_out has None, that receiver is skipped)."""
    bind_dequantize(qu, codes, scales, rest, full_out)(stream)


def bind_quantize_rows(x, codes, scales, channel=None, offsets=None):
    """fsdp_quantize_rows with cached arguments; call as f(stream=None)."""
    px, pc = _matrix(x, "x"), _codes(codes, "codes")
    if tuple(codes.shape) != tuple(x.shape):
        raise ValueError("codes must have x's shape")
    rows, cols = x.shape
    if codes.data_ptr() % 16 or _pitch(codes, "codes") % 16:
        raise ValueError("rows of codes must begin at multiples of 16 bytes")
    groups, ch = 1, None
    if channel is not None:
        groups = channel.shape[0] if channel.dim() == 2 else 1
        ch = _scales(channel, "channel", groups * cols)
    off = _offsets(offsets, groups if channel is not None or offsets is None
                   else offsets.numel() - 1)
    if channel is None and offsets is not None:
        groups = offsets.numel() - 1
    tensors = [t for t in (x, codes, scales, channel, offsets) if t is not None]
    args = (px, _dtype_code(x), rows, cols, _row_stride(x, "x"), ch, cols, off, groups, pc,
            _pitch(codes, "codes"), _scales(scales, "scales", rows))
    return _bound("fsdp_quantize_rows", args, tensors, tensors)


def fsdp_quantize_rows(x, codes, scales, channel=None, offsets=None, stream=None):
    """codes [rows, cols] int8 and scales [rows] of the rows of x (bf16 or fp32),
    each element first times channel [cols] (or [groups, cols] by the row's group)
    where given."""
    bind_quantize_rows(x, codes, scales, channel, offsets)(stream)
