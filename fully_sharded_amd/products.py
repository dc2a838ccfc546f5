"""The unit's matrix products: the binding of fsdp_grouped_matmul and
fsdp_grouped_matmul_i8 (see include/fsdp_mi355x.h).

Linear layers of a gathered unit, their input gradients and their weight
gradients, of one weight or of experts (rows of the activations sorted by
expert, `offsets` [groups + 1] int32 on the GPU):

    W, = plan.unflatten(recv[r])                     # [out, in] or [groups, out, in]
    fsdp_grouped_matmul("nt", x, W, y, offsets)      # y = x W^T
    fsdp_grouped_matmul("nn", dy, W, dx, offsets)    # dx = dy W
    dW, = plan.unflatten(grads[r])
    fsdp_grouped_matmul("tn", dy, x, dW, offsets)    # dW = dy^T x

For weights [in, out] these are "nn", "nt", and "tn" of x with dy.

Tensors are matrices with rows anywhere (stride of the last dimension 1);
weights may have a leading dimension of groups.  Every call runs on the GPU
that holds its tensors, which has to be the current one, and on the current
stream unless another is given; tensors of a call on another stream have to
live until it is done there, and the caller orders it with what else writes and
reads them.  The bind_* forms check the tensors and marshal the pointers once,
for loops.
"""

from __future__ import annotations

import ctypes

import torch

from . import binding as _b
from .binding import MatmulShape, _check, _dtype_code, lib
from .muon import _bound

_OPS = {"nt": 0, "nn": 1, "tn": 2}


def _matrix(t, what, dims=(2,)):
    """Pointer, shape and strides of a matrix (or a stack of them)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what} must be a GPU tensor")
    if t.dim() not in dims:
        raise ValueError(f"{what} must have {' or '.join(map(str, dims))} dimensions")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what}'s rows must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _row_stride(t, what):
    """Elements from one row to the next; rows that follow each other where
    there is only one."""
    rows, cols = t.shape[-2], t.shape[-1]
    if rows <= 1:
        return max(cols, 1)
    if t.stride(-2) < cols:
        raise ValueError(f"{what}'s rows overlap")
    return t.stride(-2)


def _offsets(offsets, groups):
    if offsets is None:
        if groups != 1:
            raise ValueError("more than one group needs offsets")
        return None
    if not isinstance(offsets, torch.Tensor) or not offsets.is_cuda or \
            offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous int32 GPU tensor of one dimension")
    if offsets.numel() != groups + 1:
        raise ValueError("offsets must have groups + 1 elements")
    return ctypes.c_void_p(offsets.data_ptr())


def _groups(t):
    return t.shape[0] if t.dim() == 3 else 1


def _shape(op, a, b, c, accumulate):
    """MatmulShape of a call, its tensors' shapes checked against each other."""
    if op not in _OPS:
        raise ValueError(f"op is one of {sorted(_OPS)}")
    stacked = c if op == "tn" else b
    for t, what in ((a, "a"), (b, "b"), (c, "c")):
        _matrix(t, what, (2, 3) if t is stacked else (2,))
    rows, groups = a.shape[0], _groups(stacked)
    if op == "tn":
        n, k = a.shape[1], b.shape[1]
        ok = b.shape[0] == rows and tuple(c.shape[-2:]) == (n, k)
    else:
        k = a.shape[1]
        n = b.shape[-2] if op == "nt" else b.shape[-1]
        ok = b.shape[-1 if op == "nt" else -2] == k and tuple(c.shape) == (rows, n)
    if not ok:
        raise ValueError(f"{op}: the shapes {tuple(a.shape)}, {tuple(b.shape)} and "
                         f"{tuple(c.shape)} do not fit")
    stride = stacked.stride(0) if groups > 1 else 0
    return MatmulShape(_OPS[op], groups, rows, n, k, _row_stride(a, "a"), _row_stride(b, "b"),
                       _row_stride(c, "c"), stride, int(bool(accumulate)), 0)


def _workspace_bytes(shape, dtype):
    n = ctypes.c_int64()
    _check("fsdp_grouped_matmul_workspace",
           lib().fsdp_grouped_matmul_workspace(ctypes.byref(shape), dtype, ctypes.byref(n)))
    return n.value


def grouped_matmul_workspace(op, a, b, c):
    """A workspace for this product, or None where it needs none."""
    return _workspace_for(op, a, b, c, None)


def _workspace_for(op, a, b, c, stream):
    """grouped_matmul_workspace for a call on `stream` (None: the current one).
    Memory that the allocator hands out may still be in use by work of the
    stream that it is allocated on, so that is the stream that will use it."""
    n = _workspace_bytes(_shape(op, a, b, c, False), _dtype_code(a))
    if not n or stream is None:
        return torch.empty(n, dtype=torch.uint8, device=a.device) if n else None
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_b._stream(stream).value or 0)
    with torch.cuda.stream(stream):
        return torch.empty(n, dtype=torch.uint8, device=a.device)


def _plain(op, a, b, c, offsets, accumulate, workspace):
    """(arguments, what they point to, the tensors)."""
    shape = _shape(op, a, b, c, accumulate)
    dt = _dtype_code(a)
    if _dtype_code(b) != dt:
        raise ValueError("a and b must have one dtype")
    out = _dtype_code(c)
    off = _offsets(offsets, shape.groups)
    ws, n = None, 0
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8:
            raise ValueError("the workspace is a uint8 tensor")
        ws, n = ctypes.c_void_p(_b._dev(workspace, "workspace")), workspace.numel()
    tensors = [t for t in (a, b, c, offsets, workspace) if t is not None]
    args = (ctypes.byref(shape), off, _matrix(a, "a"), _matrix(b, "b", (2, 3)), dt,
            _matrix(c, "c", (2, 3)), out, ws, n)
    return args, (shape, *tensors), tensors


def bind_grouped_matmul(op: str, a, b, c, offsets=None, accumulate: bool = False,
                        workspace=None):
    """fsdp_grouped_matmul with cached arguments; call as f(stream=None).  A
    workspace that is needed and not given is allocated and kept, and the
    binding waits for the current stream, whose work may still use that memory
    (bound while that stream is captured it does not: such a workspace is the
    graph's): so any stream may use it, but calls of one binding that may
    overlap in time, on two streams or in replays of two captured graphs, race
    on it."""
    given = workspace
    if given is None:
        workspace = grouped_matmul_workspace(op, a, b, c)
        if workspace is not None and not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(a.device).synchronize()
    args, keep, tensors = _plain(op, a, b, c, offsets, accumulate, workspace)
    bound = _bound("fsdp_grouped_matmul", args, keep, tensors)
    if given is not None or workspace is None:
        return bound
    current, device = torch._C._cuda_getCurrentRawStream, a.device.index
    known = {current(device)}

    def run(stream=None):
        bound(stream)
        handle = current(device) if stream is None else _b._stream(stream).value or 0
        if handle not in known:
            # the allocator may hand the workspace out again, once nobody has the
            # binding, only when this call is done
            workspace.record_stream(torch.cuda.ExternalStream(handle))
            known.add(handle)
    run.call = bound.call
    return run


def fsdp_grouped_matmul(op: str, a, b, c, offsets=None, accumulate: bool = False,
                        workspace=None, stream=None):
    """The product of bf16 or fp32 matrices into c (bf16 or fp32), by groups of
    rows where offsets are given:
      "nt"  c[t] = a[t] b_g^T      "nn"  c[t] = a[t] b_g
      "tn"  c_g = a[rows of g]^T b[rows of g]
    accumulate: added to what c holds."""
    if workspace is None:
        workspace = _workspace_for(op, a, b, c, stream)
    args, keep, tensors = _plain(op, a, b, c, offsets, accumulate, workspace)
    _bound("fsdp_grouped_matmul", args, keep, tensors)(stream)


def _codes(t, what, dims=(2,)):
    """A matrix of codes: rows at multiples of 16 bytes, readable to the next."""
    p = _matrix(t, what, dims)
    if t.dtype != torch.int8:
        raise ValueError(f"{what} must be int8")
    if t.numel():
        last = t.storage_offset() + sum((n - 1) * s for n, s in zip(t.shape[:-1], t.stride()[:-1]))
        if last + -(-t.shape[-1] // 16) * 16 > t.untyped_storage().nbytes():
            raise ValueError(f"{what}'s last row must be readable to a multiple of 16 bytes")
    return p


def _pitch(t, what):
    """Bytes from one row of codes to the next."""
    return -(-t.shape[-1] // 16) * 16 if t.shape[-2] <= 1 else _row_stride(t, what)


def _scales(t, what, n):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32 or \
            not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{what} must be a contiguous fp32 GPU tensor of {n} elements")
    return ctypes.c_void_p(t.data_ptr())


def bind_grouped_matmul_i8(op: str, a, a_scale, b, b_scale, c, offsets=None,
                           accumulate: bool = False):
    """fsdp_grouped_matmul_i8 with cached arguments; call as f(stream=None)."""
    if op not in ("nt", "nn"):
        raise ValueError("op is one of ['nn', 'nt']")
    shape = _shape(op, a, b, c, accumulate)
    pa, pb = _codes(a, "a"), _codes(b, "b", (2, 3))
    shape.lda, shape.ldb = _pitch(a, "a"), _pitch(b, "b")
    sa = _scales(a_scale, "a_scale", shape.rows)
    sb = None
    if b_scale is not None:
        sb = _scales(b_scale, "b_scale", shape.groups * shape.n)
    off = _offsets(offsets, shape.groups)
    tensors = [t for t in (a, a_scale, b, b_scale, c, offsets) if t is not None]
    args = (ctypes.byref(shape), off, pa, sa, pb, sb, shape.n, _matrix(c, "c"), _dtype_code(c))
    return _bound("fsdp_grouped_matmul_i8", args, (shape, *tensors), tensors)


def fsdp_grouped_matmul_i8(op: str, a, a_scale, b, b_scale, c, offsets=None,
                           accumulate: bool = False, stream=None):
    """The product of 8-bit codes (-127 to 127; -128 too where the sum has at most
    131,071 terms) into c (bf16 or fp32), "nt" or "nn" as in
    fsdp_grouped_matmul, times a_scale [rows] and b_scale [groups, n] (None: no
    such factor).  accumulate: added to what c holds."""
    bind_grouped_matmul_i8(op, a, a_scale, b, b_scale, c, offsets, accumulate)(stream)
