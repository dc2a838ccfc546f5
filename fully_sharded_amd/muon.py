"""The Muon optimiser on a unit's matrices: the binding of the library's
fsdp_muon_* calls and fsdp_orthogonalize (see include/fsdp_mi355x.h).

A step of one unit, by its parts:

    mu = Muon(plan, [0, 1, 2])                  # which parameters are its matrices
    fsdp_muon_momentum(mu, hp, grads, m, update)         # shards -> gathered update
    fsdp_orthogonalize(mu, hp, update, ortho, workspace)
    fsdp_muon_apply(mu, hp, ortho, master, param)        # back on the shards

or as one call, with AdamW on the unit's other parameters:

    fsdp_muon_shard_step(mu, hp, grads, master, m, param, workspace,
                         adamw=ADAMW, step=t, v=v)

Hyper-parameters are a dict like MUON.  Every call runs on the GPU that holds
its tensors, which has to be the current one, and on the current stream
unless another is given; tensors and workspaces of a call on another stream
have to live until it is done there.  The bind_* forms check the tensors and
marshal the pointers once, for loops, the hyper-parameters with them.
"""

from __future__ import annotations

import ctypes
import sys

import torch

from . import binding as _b
from .binding import (AdamWHParams, BoundCall, MuonHParams, Plan, _check, _dev, _dtype_code,
                      _items, _ptr_array, _stream, lib)

#: The usual hyper-parameters.  coefficients: (a, b, c) of one step
#: a x + b x^3 + c x^5; scale: "none", "aspect" (sqrt(max(1, rows / columns)))
#: or "rms" (0.2 sqrt(max(rows, columns))).
MUON = {"lr": 1e-3, "momentum": 0.95, "weight_decay": 0.01, "eps": 1e-7,
        "coefficients": (3.4445, -4.7750, 2.0315), "steps": 5, "nesterov": True, "scale": "rms"}

_SCALES = {"none": 0, "aspect": 1, "rms": 2}


def _hp(hp: dict) -> MuonHParams:
    a, b, c = hp["coefficients"]
    if hp["scale"] not in _SCALES:
        raise ValueError(f"scale is one of {sorted(_SCALES)}")
    return MuonHParams(hp["lr"], hp["momentum"], hp["weight_decay"], hp["eps"], a, b, c,
                       int(hp["steps"]), int(bool(hp["nesterov"])), _SCALES[hp["scale"]])


def _on_current_device(*tensors):
    """The library works on the current device: tensors elsewhere are refused."""
    for t in tensors:
        if t.device.index != torch.cuda.current_device():
            raise ValueError(f"a tensor is on {t.device}, the current device is "
                             f"cuda:{torch.cuda.current_device()}")


class Muon:
    """The parameters of `plan` that Muon updates (their indices; by default
    every parameter of two dimensions or more)."""

    def __init__(self, plan: Plan, params=None):
        if params is None:
            params = [p for p, s in enumerate(plan.shapes) if len(s) >= 2]
        params = [int(p) for p in params]
        arr = (ctypes.c_int32 * max(1, len(params)))(*params)
        h = ctypes.c_void_p()
        _check("fsdp_muon_plan", lib().fsdp_muon_plan(plan.handle, len(params), arr,
                                                      ctypes.byref(h)))
        self._h = h
        self.plan = plan
        self.params = params

    @property
    def handle(self):
        return self._h

    def __del__(self):
        # at interpreter exit the HIP runtime may already be gone: leak then
        h = getattr(self, "_h", None)
        if h is not None and _b._lib is not None and not sys.is_finalizing():
            _b._lib.fsdp_muon_destroy(h)
            self._h = None

    def prepare(self, stream=None):
        """Upload the work tables to the current device now."""
        _check("fsdp_muon_prepare", lib().fsdp_muon_prepare(self._h, _stream(stream)))

    def workspace_bytes(self, update_dtype=torch.bfloat16, ortho_dtype=torch.bfloat16):
        """(bytes of fsdp_orthogonalize's workspace, bytes of
        fsdp_muon_shard_step's)."""
        def code(dtype):
            return _dtype_code(torch.empty(0, dtype=dtype))
        one, step = ctypes.c_int64(), ctypes.c_int64()
        _check("fsdp_muon_workspace",
               lib().fsdp_muon_workspace(self._h, code(update_dtype), code(ortho_dtype),
                                         ctypes.byref(one), ctypes.byref(step)))
        return one.value, step.value

    def workspace(self, update_dtype=torch.bfloat16, ortho_dtype=torch.bfloat16, device="cuda"):
        """A workspace for fsdp_orthogonalize with these types."""
        return torch.empty(self.workspace_bytes(update_dtype, ortho_dtype)[0],
                           dtype=torch.uint8, device=device)

    def step_workspace(self, device="cuda"):
        """A workspace for fsdp_muon_shard_step."""
        return torch.empty(self.workspace_bytes()[1], dtype=torch.uint8, device=device)

    def work_items(self, space: int):
        """Host copy of the per-element work items: list of (dst, src, len);
        space 0 = shard space (apply), 1 = flat space (momentum)."""
        return _items(lambda out, cap, n: lib().fsdp_muon_work_items(self._h, space, out, cap, n),
                      "fsdp_muon_work_items")


def fsdp_muon_plan(plan: Plan, params=None) -> Muon:
    return Muon(plan, params)


def _full(mu, t, what):
    if t.numel() != mu.plan.T:
        raise ValueError(f"{what} must have T elements")
    return ctypes.c_void_p(_dev(t, what))


def _shards(mu, t, what, fp32=True):
    if t.numel() != mu.plan.R * mu.plan.S or (fp32 and t.dtype != torch.float32):
        raise ValueError(f"{what} must {'be fp32 with' if fp32 else 'have'} R*S elements")
    return ctypes.c_void_p(_dev(t, what))


def _grads(mu, grads, replicas):
    """(pointers, dtype, the tensors) of R replicas or of one reduced tensor."""
    plan = mu.plan
    if not replicas:
        if isinstance(grads, (list, tuple)):
            (grads,) = grads
        if grads.numel() != plan.R * plan.S or grads.dtype != torch.float32:
            raise ValueError("the reduced gradient must be fp32 with R*S elements")
        return _ptr_array([grads], "grads"), _b.F32, [grads]
    grads = list(grads)
    if len(grads) != plan.R:
        raise ValueError("need R gradient replicas")
    dt = _dtype_code(grads[0])
    for g in grads:
        if g.numel() != plan.T or _dtype_code(g) != dt:
            raise ValueError("gradient size or dtype mismatch")
    return _ptr_array(grads, "grads"), dt, grads


def _work(t):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8:
        raise ValueError("the workspace is a uint8 tensor")
    return ctypes.c_void_p(_dev(t, "workspace")), t.numel()


def _caller(name, keep, tensors):
    """(BoundCall, f(args, stream)): the library call on the given stream, or
    on the current one of the tensors' device, which has to be the current
    device at every call and the given stream's.  The handle is asked of torch directly: a Stream
    object costs 2.7 us, a third of a small call."""
    _on_current_device(*tensors)
    device = tensors[0].device.index
    call = BoundCall(name, None, keep)
    fn, current, raw = call._fn, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream

    def go(args, stream):
        if current() != device:
            raise ValueError(f"the tensors are on cuda:{device}, the current device is "
                             f"cuda:{current()}")
        of = getattr(stream, "device", None)  # (a ctypes handle does not say whose it is)
        if of is not None and of.index != device:
            raise ValueError(f"the tensors are on cuda:{device}, the stream on {of}")
        status = fn(*args, raw(device) if stream is None else _stream(stream))
        if status != 0:
            _check(name, status)
    return call, go


def _bound(name, args, keep, tensors):
    call, go = _caller(name, keep, tensors)

    def run(stream=None):
        go(args, stream)
    run.call = call
    return run


def bind_muon_momentum(mu: Muon, hp: dict, grads, m, update, grads_are_replicas: bool = True):
    """fsdp_muon_momentum with cached arguments; call as f(stream=None)."""
    h = _hp(hp)
    arr, dt, gs = _grads(mu, grads, grads_are_replicas)
    args = (mu.handle, ctypes.byref(h), arr, dt, int(bool(grads_are_replicas)),
            _shards(mu, m, "m"), _full(mu, update, "update"), _dtype_code(update))
    return _bound("fsdp_muon_momentum", args, (mu, h, gs, m, update), (*gs, m, update))


def fsdp_muon_momentum(mu: Muon, hp: dict, grads, m, update, grads_are_replicas: bool = True,
                       stream=None):
    """Mean of the R replicas [T] (or, with grads_are_replicas=False, one
    reduced fp32 [R*S] tensor), the momentum's shards m [R*S] in place, and
    the gathered update [T]."""
    bind_muon_momentum(mu, hp, grads, m, update, grads_are_replicas)(stream)


def bind_orthogonalize(mu: Muon, hp: dict, update, ortho, workspace):
    """fsdp_orthogonalize with cached arguments; call as f(stream=None)."""
    h = _hp(hp)
    ws, n = _work(workspace)
    args = (mu.handle, ctypes.byref(h), _full(mu, update, "update"), _dtype_code(update),
            _full(mu, ortho, "ortho"), _dtype_code(ortho), ws, n)
    return _bound("fsdp_orthogonalize", args, (mu, h, update, ortho, workspace),
                  (update, ortho, workspace))


def fsdp_orthogonalize(mu: Muon, hp: dict, update, ortho, workspace, stream=None):
    """Newton-Schulz products on every matrix of update [T] into ortho [T]
    (which may be update itself)."""
    bind_orthogonalize(mu, hp, update, ortho, workspace)(stream)


def bind_muon_apply(mu: Muon, hp: dict, ortho, master, param_out):
    """fsdp_muon_apply with cached arguments; call as f(stream=None)."""
    h = _hp(hp)
    args = (mu.handle, ctypes.byref(h), _full(mu, ortho, "ortho"), _dtype_code(ortho),
            _shards(mu, master, "master"), _shards(mu, param_out, "param_out", False),
            _dtype_code(param_out))
    return _bound("fsdp_muon_apply", args, (mu, h, ortho, master, param_out),
                  (ortho, master, param_out))


def fsdp_muon_apply(mu: Muon, hp: dict, ortho, master, param_out, stream=None):
    """master [R*S] <- master (1 - lr wd) - lr scale ortho, and its recast."""
    bind_muon_apply(mu, hp, ortho, master, param_out)(stream)


def bind_muon_shard_step(mu: Muon, hp: dict, grads, master, m, param_out, workspace,
                         adamw: dict | None = None, v=None):
    """fsdp_muon_shard_step with cached arguments; call as f(step,
    stream=None), step being AdamW's counter."""
    h = _hp(hp)
    if (adamw is None) != (v is None):
        raise ValueError("AdamW on the other parameters needs its hyper-parameters and v")
    a = None if adamw is None else AdamWHParams(adamw["lr"], adamw["beta1"], adamw["beta2"],
                                                adamw["eps"], adamw["weight_decay"])
    arr, dt, gs = _grads(mu, grads, True)
    ws, n = _work(workspace)
    head = (mu.handle, ctypes.byref(h), None if a is None else ctypes.byref(a))
    tail = (arr, dt, _shards(mu, master, "master"), _shards(mu, m, "m"),
            None if v is None else _shards(mu, v, "v"),
            _shards(mu, param_out, "param_out", False), _dtype_code(param_out), ws, n)
    state = (master, m, param_out, workspace) + (() if v is None else (v,))
    call, go = _caller("fsdp_muon_shard_step", (mu, h, a, gs, state), (*gs, *state))

    def run(step=1, stream=None):
        go((*head, int(step), *tail), stream)
    run.call = call
    return run


def fsdp_muon_shard_step(mu: Muon, hp: dict, grads, master, m, param_out, workspace,
                         adamw: dict | None = None, step: int = 1, v=None, stream=None):
    """One optimiser step of a unit from its R gradient replicas: Muon on the
    chosen matrices and, with adamw given, AdamW (step counter `step`) on all
    its other parameters."""
    bind_muon_shard_step(mu, hp, grads, master, m, param_out, workspace, adamw, v)(step, stream)
