"""The AdamW step over many tensors in one launch, and the norm of their gradients.

    opt = AdamW(params, lr=3e-4, weight_decay=0.1, state_bits=8)
    ws = grad_norm_workspace(grads)
    norm, scale = grad_norm(grads, max_norm=1.0, ws=ws)
    opt.step(grads, grad_scale=scale)

Parameters are bf16 or fp32, gradients either; states fp32 or 8 bits (e4m3 with a
scale for each 128 elements, rounded stochastically).  A bf16 parameter has an
fp32 master copy (master=True) or is rounded stochastically.  The kernels run in
libglr_moe.so (include/moe.h: moe_adamw, moe_grad_norm)."""
from __future__ import annotations

import ctypes
import math
import operator
from typing import Optional

import numpy as np
import torch

from . import _lib
from .moe import SizedWorkspace, _need, _on, _opt, _sized

_BF16, _F32 = torch.bfloat16, torch.float32
_TYPES = {_BF16, _F32}


_FIELDS = np.dtype([(name, np.uint64) for name in ("p", "g", "master", "m", "v", "m_scale", "v_scale")] +
                   [("n", np.int64), ("weight_decay", np.float64), ("ordinal", np.uint32), ("flags", np.int32)])


def _table(n: int):
    """(ctypes array of n tensors, the same memory's fields as numpy columns)."""
    table = (_lib.AdamwTensor * max(n, 1))()
    return table, np.frombuffer(table, dtype=_FIELDS)


def _check_tensors(tensors, name, device):
    for i, t in enumerate(tensors):
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s[%d] must be a tensor" % (name, i))
        if t.dtype not in _TYPES:
            raise TypeError("%s[%d] must be torch.bfloat16 or torch.float32, got %s" % (name, i, t.dtype))
        if t.device != device:
            raise ValueError("%s[%d] must be on %s, got %s" % (name, i, device, t.device))
        if not t.is_contiguous():
            raise ValueError("%s[%d] must be contiguous" % (name, i))


_address, _contiguous, _where = torch.Tensor.data_ptr, torch.Tensor.is_contiguous, torch.Tensor.get_device
_type = operator.attrgetter("dtype")
_shape = operator.attrgetter("shape")


def _refuse_overlaps(named) -> None:
    """Lists of (name, contiguous tensors or Nones) of which no two may share memory: the
    kernel's blocks read and write all of them at once."""
    spans = sorted((t.data_ptr(), t.numel() * t.element_size(), name, i) for name, held in named
                   for i, t in enumerate(held) if t is not None and t.numel())
    for (a, size, *first), (b, _, *second) in zip(spans, spans[1:]):
        if a + size > b:
            raise ValueError("%s[%d] and %s[%d] overlap" % (*first, *second))


def _addresses_of(tensors) -> list:
    try:
        return list(map(_address, tensors))
    except TypeError:                            # (a master that is None, beside an fp32 parameter)
        return [t.data_ptr() if isinstance(t, torch.Tensor) else None for t in tensors]


def _fill_grads(grads, table, device):
    """Checks the gradients, puts their addresses into a table and gives the flags of
    their types.  (Hundreds of small tensors: an attribute at a time over all.)"""
    n = len(grads)
    try:
        types = list(map(_type, grads))
        same = types[0] if types.count(types[0]) == n else None
        where = list(map(_where, grads))
        plain = (all(map(_contiguous, grads)) and where.count(device.index) == n and
                 (same in _TYPES if same is not None else set(types) <= _TYPES))
        if plain:
            table["g"][:n] = np.fromiter(map(_address, grads), np.uint64, n)
    except (AttributeError, TypeError):
        plain = False
    if not plain:
        _check_tensors(grads, "grads", device)
        raise ValueError("gradients that cannot be read")
    if same is not None:
        return _lib.MOE_ADAMW_GRAD_BF16 if same == _BF16 else 0
    return np.array([_lib.MOE_ADAMW_GRAD_BF16 if t == _BF16 else 0 for t in types], np.int32)


def grad_norm_workspace(grads, device=None) -> SizedWorkspace:
    """The workspace of grad_norm over this many gradients."""
    if device is None and len(grads):
        device = grads[0].device
    return SizedWorkspace(_lib.load().moe_grad_norm_workspace_bytes(len(grads)), "moe_grad_norm", device)


def grad_norm(grads, max_norm: float = 1.0, *, ws: Optional[SizedWorkspace] = None, out=None):
    """moe_grad_norm: (norm [1], scale [1]) fp32: the 2-norm over all gradients, and
    what they are to be multiplied by so that it is at most max_norm (NaN where the
    norm is not finite: AdamW.step then writes nothing)."""
    grads = list(grads)
    if not grads:
        raise ValueError("grad_norm needs a gradient")
    if not isinstance(grads[0], torch.Tensor):
        raise TypeError("grads[0] must be a tensor")
    dev = grads[0].device
    table, cols = _table(len(grads))
    cols["flags"] = _fill_grads(grads, cols, dev)
    cols["n"] = np.fromiter(map(torch.Tensor.numel, grads), np.int64, len(grads))
    norm, scale = out if out is not None else (torch.empty(1, dtype=_F32, device=dev),
                                               torch.empty(1, dtype=_F32, device=dev))
    pn = _need(norm, "norm", _F32, (1,), dev)
    ps = _need(scale, "scale", _F32, (1,), dev)
    lib = _lib.load()
    ws = _sized(ws, int(lib.moe_grad_norm_workspace_bytes(len(grads))), "moe_grad_norm", dev)
    _lib.check(_on(dev, lib.moe_grad_norm, len(grads), ctypes.addressof(table), max_norm, pn, ps, ws.ptr, ws.nbytes),
               "moe_grad_norm")
    return norm, scale


class AdamW:
    """AdamW over `params` (contiguous bf16 or fp32 tensors, which the steps change in
    place; no two of them, or of the states, may share memory).

    weight_decay: one for all, or one for each.  state_bits: 32 (m and v in fp32) or
    8 (m and sqrt(v) in e4m3 with scales for each 128 elements).  master: keep fp32
    copies of bf16 parameters; without, they are rounded stochastically.  seed: of
    the random bits.  state: dict of lists (m, v, with 8 bits m_scale and v_scale,
    with master master: None for fp32 parameters) to continue from after `step`
    steps, used in place; without, the state of no step is made.  A step works on the
    tensors that `params` and `state` hold then: others may take their places (the
    replaced ones are let go by the next step).

    capturable=True keeps the step's number and lr in tensors on the device
    (step_count [1] int64, lr_now [1] fp32), which each step() advances and reads
    there, so that a captured step goes on counting as it is replayed."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.01, *,
                 state_bits: int = 32, master: bool = False, seed: int = 0, step: int = 0, state: Optional[dict] = None,
                 capturable: bool = False):
        self.params = list(params)
        if not self.params:
            raise ValueError("AdamW needs a parameter")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32, got %r" % (state_bits,))
        if not isinstance(self.params[0], torch.Tensor):
            raise TypeError("params[0] must be a tensor")
        self.device = dev = self.params[0].device
        _check_tensors(self.params, "params", dev)
        betas = tuple(betas)
        if not math.isfinite(lr):
            raise ValueError("lr must be finite, got %r" % (lr,))
        if len(betas) != 2 or not all(0.0 <= b < 1.0 for b in betas):
            raise ValueError("betas must be two numbers from 0 and below 1, got %r" % (betas,))
        if not 0.0 <= eps < math.inf:
            raise ValueError("eps must be finite and at least 0, got %r" % (eps,))
        if step < 0:
            raise ValueError("step must be at least 0, got %r" % (step,))
        n = len(self.params)
        decay = list(weight_decay) if hasattr(weight_decay, "__len__") else [weight_decay] * n
        if len(decay) != n:
            raise ValueError("weight_decay must be a number or %d of them, got %d" % (n, len(decay)))
        if not all(0.0 <= d < math.inf for d in decay):
            raise ValueError("weight_decay must be finite and at least 0, got %r" % (weight_decay,))
        self.lr, self.betas, self.eps, self.step_number, self.seed = lr, betas, eps, step, seed
        self.state_bits, self.master = state_bits, master
        self._sizes = [p.numel() for p in self.params]
        self._shapes = [p.shape for p in self.params]
        self.state = self._new_state() if state is None else state
        names = ["m", "v"] + (["m_scale", "v_scale"] if state_bits == 8 else []) + (["master"] if master else [])
        self._names, self._decay = names, [float(d) for d in decay]
        self._fill_table()
        self._cfg = _lib.AdamwCfg(lr, self.betas[0], self.betas[1], eps, max(step, 1), seed & 0xffffffff, 0)
        self.step_count = self.lr_now = None
        if capturable:
            self.step_count = torch.tensor([step], dtype=torch.int64, device=dev)
            self.lr_now = torch.tensor([lr], dtype=_F32, device=dev)
        self.last_launches = 0

    def _fill_table(self) -> None:
        """The library's table of the parameters and their states (all of it, or with an
        error what it was)."""
        n, dev, bits = len(self._sizes), self.device, self.state_bits
        for name, held in [("params", self.params)] + [("state[%r]" % (s,), self.state[s]) for s in self._names]:
            if len(held) != n:
                raise ValueError("%s must have %d tensors, got %d" % (name, n, len(held)))
        _check_tensors(self.params, "params", dev)
        table, cols = _table(n)
        for i, p in enumerate(self.params):
            size = self._sizes[i]
            if p.shape != self._shapes[i]:
                raise ValueError("params[%d] must have shape %s, got %s" % (i, tuple(self._shapes[i]), tuple(p.shape)))
            t = table[i]
            t.p, t.n, t.weight_decay, t.ordinal = p.data_ptr(), size, self._decay[i], i
            kind = torch.float8_e4m3fn if bits == 8 else _F32
            for name in self._names:
                s, what = self.state[name][i], "state[%r][%d]" % (name, i)
                if name in ("m", "v"):
                    setattr(t, name, _need(s, what, kind, (size,), dev))
                elif name != "master":
                    setattr(t, name, _need(s, what, torch.float8_e8m0fnu, (-(-size // 128),), dev))
                elif p.dtype == _BF16:
                    t.master = _need(s, what, _F32, (size,), dev)
            t.flags = (_lib.MOE_ADAMW_STATES_IN_BYTES if bits == 8 else 0) | \
                      (_lib.MOE_ADAMW_PARAM_BF16 if p.dtype == _BF16 else 0)
        _refuse_overlaps([("params", self.params)] + [("state[%r]" % (s,), self.state[s]) for s in self._names])
        self._table, self._cols, self._flags = table, cols, cols["flags"][:n].copy()
        # (kept, so that nothing else is given a replaced tensor's memory, and with it an
        # address that step() knows, before step() has looked)
        self._held = self._tensors()
        self._addresses = _addresses_of(self._held)

    def _tensors(self) -> list:
        """The parameters' and states' tensors as they are now."""
        held = [*self.params]
        for name in self._names:
            held += self.state[name]
        return held

    def _new_state(self) -> dict:
        dev, sizes = self.device, self._sizes
        if self.state_bits == 32:
            s = {name: [torch.zeros(n, dtype=_F32, device=dev) for n in sizes] for name in ("m", "v")}
        else:
            s = {name: [torch.zeros(n, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for n in sizes]
                 for name in ("m", "v")}
            for name in ("m_scale", "v_scale"):
                s[name] = [torch.full((-(-n // 128),), 127, dtype=torch.uint8, device=dev).view(torch.float8_e8m0fnu)
                           for n in sizes]
        if self.master:
            s["master"] = [p.detach().reshape(-1).float() if p.dtype == _BF16 else None for p in self.params]
        return s

    def step(self, grads, *, lr: Optional[float] = None, grad_scale=None) -> None:
        """One step with the gradients of the parameters, in their order (contiguous,
        bf16 or fp32, of the parameters' shapes); lr from now on, if given;
        grad_scale [1] fp32 on the device: what the gradients are multiplied by (not
        finite: nothing is written, though the step counts)."""
        grads = list(grads)
        if _addresses_of(self._tensors()) != self._addresses:        # (one of them has other memory)
            self._fill_table()
        if len(grads) != len(self._sizes):
            raise ValueError("%d gradients expected, got %d" % (len(self._sizes), len(grads)))
        bits = _fill_grads(grads, self._cols, self.device)
        if list(map(_shape, grads)) != self._shapes:
            i = next(i for i, (g, s) in enumerate(zip(grads, self._shapes)) if g.shape != s)
            raise ValueError("grads[%d] must have shape %s, got %s" % (i, tuple(self._shapes[i]), tuple(grads[i].shape)))
        self._cols["flags"] = self._flags | bits
        ps = _opt(grad_scale, "grad_scale", _F32, (1,), self.device)
        new_lr = self.lr if lr is None else lr
        if not math.isfinite(new_lr):
            raise ValueError("lr must be finite, got %r" % (new_lr,))
        cfg = self._cfg
        cfg.lr, cfg.step = new_lr, self.step_number + 1
        pc = pl = None
        if self.step_count is not None:
            if lr is not None:
                self.lr_now.fill_(lr)
            self.step_count.add_(1)
            pc, pl = self.step_count.data_ptr(), self.lr_now.data_ptr()
        try:
            _lib.check(_on(self.device, _lib.load().moe_adamw, len(grads), ctypes.addressof(self._table), ctypes.byref(cfg),
                           ps, pc, pl), "moe_adamw")
        except Exception:                        # (what the kernel would have read counts no step either)
            if self.step_count is not None:
                self.step_count.sub_(1)
                if lr is not None:
                    self.lr_now.fill_(self.lr)
            raise
        self.lr = new_lr
        self.step_number += 1
        self.last_launches = _lib.load().moe_last_launch_count()
