"""PyTorch-facing calls of the GB300 MoE layer forward.

Each function checks tensor shapes, dtypes and devices, passes raw pointers
and the current CUDA stream to the C ABI (include/moe.h) and returns torch
tensors.  No arithmetic of the layer happens here: routing, bucketing, the
expert GEMMs and the combine all run in libglr_moe.so's kernels.

The layer is the one of the article "InternLumina-U2中256个专家的路由秘密：
分组受限Top-K、Expert Bias与Fused MoE详解": fp32 sigmoid router over E experts,
group-limited top-k (section 二), selection-only expert bias (section 三),
SwiGLU experts with stacked [E, I, H] weights (section 四) and one shared
expert (section 五).
"""
from __future__ import annotations

import ctypes
import functools
import types
import dataclasses
from typing import Optional

import torch

from . import _lib


@dataclasses.dataclass(frozen=True)
class MoeConfig:
    """moe_cfg of include/moe.h (defaults: the article's hyper-parameter table)."""
    T: int
    H: int = 2048
    E: int = 256
    n_group: int = 8
    topk_group: int = 4
    k: int = 8
    I: int = 512
    Is: int = 512
    rsf: float = 2.5
    eps: float = 1e-20

    def c(self) -> _lib.MoeCfg:
        """A new structure of these fields, the caller's own."""
        return _lib.MoeCfg(self.T, self.H, self.E, self.n_group, self.topk_group, self.k, self.I, self.Is, self.rsf,
                           self.eps)

    def ref(self):
        """A pointer for the library's calls, which take it as const (made once per
        configuration: the fields never change)."""
        r = self.__dict__.get("_ref")
        if r is None:
            r = ctypes.byref(self.c())
            object.__setattr__(self, "_ref", r)
        return r

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "_ref"}

    def with_T(self, T: int) -> "MoeConfig":
        return dataclasses.replace(self, T=T)


# workspace kind of moe_layer (a tag of this module; its size also depends on flags)
WS_LAYER = 3


def workspace_bytes(cfg: MoeConfig, which: int, flags: int = 0) -> int:
    if which == WS_LAYER:
        n = _lib.load().moe_layer_workspace_bytes(cfg.ref(), flags)
    else:
        n = _lib.load().moe_workspace_bytes(cfg.ref(), which)
    if n == 0:
        raise ValueError("configuration not supported: %r" % (cfg,))
    return int(n)


class Workspace:
    """A device workspace for moe_route (ROUTE), moe_forward (FORWARD),
    moe_backward (BACKWARD) or moe_layer (WS_LAYER, sized for `flags`)."""

    def __init__(self, cfg: MoeConfig, which: int, device=None, flags: int = 0):
        self.which = which
        self.flags = flags
        self.nbytes = workspace_bytes(cfg, which, flags)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device or "cuda")
        assert self.buf.data_ptr() % 256 == 0
        _lib.check(_lib.load().moe_workspace_init(self.ptr, self.nbytes, _stream(self.buf.device)),
                   "moe_workspace_init")

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()

    def fits(self, cfg: MoeConfig, flags: Optional[int] = None) -> bool:
        return workspace_bytes(cfg, self.which, self.flags if flags is None else flags) <= self.nbytes

    def status(self, reset: bool = True) -> int:
        v = ctypes.c_int32(0)
        _lib.check(_lib.load().moe_get_status(self.ptr, self.nbytes, _stream(self.buf.device), ctypes.byref(v),
                                              1 if reset else 0), "moe_get_status")
        return int(v.value)


# the current stream's handle without a Stream object around it, where torch has
# that call (2 us less on each of the library's calls)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device) -> int:
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _need(t: torch.Tensor, name: str, dtype, shape, device) -> int:
    if (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.device == device and
            t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _opt(t, name, dtype, shape, device) -> Optional[int]:
    return None if t is None else _need(t, name, dtype, shape, device)


def _ws(ws: Optional[Workspace], cfg: MoeConfig, which: int, device) -> Workspace:
    if ws is None:
        ws = Workspace(cfg, which, device)
    elif ws.which != which or not ws.fits(cfg):
        raise ValueError("workspace of the wrong kind or too small")
    return ws


def prepare_router(cfg: MoeConfig, W_router, out=None):
    """moe_prepare_router: the exact bf16 x 3 split of the fp32 router weight,
    [3, E, H] bf16, for route(..., W_split=...)."""
    dev = W_router.device
    pw = _need(W_router, "W_router", torch.float32, (cfg.E, cfg.H), dev)
    W_split = out if out is not None else torch.empty(3, cfg.E, cfg.H, dtype=torch.bfloat16, device=dev)
    ps = _need(W_split, "W_split", torch.bfloat16, (3, cfg.E, cfg.H), dev)
    _lib.check(_lib.load().moe_prepare_router(cfg.ref(), pw, ps, _stream(dev)), "moe_prepare_router")
    return W_split


def route(cfg: MoeConfig, hidden, W_router, expert_bias=None, *, aux: bool = False,
          ws: Optional[Workspace] = None, out=None, W_split=None):
    """moe_route (or moe_route_prepared when W_split = prepare_router(W_router)
    is given): (topk_idx [T,k] int32, topk_w [T,k] fp32, expert_counts [E]
    int32, aux_P [E] fp32 or None, aux_loss [1] fp32 or None)."""
    dev = hidden.device
    ph = _need(hidden, "hidden", torch.bfloat16, (cfg.T, cfg.H), dev)
    pw = _need(W_router, "W_router", torch.float32, (cfg.E, cfg.H), dev)
    pb = _opt(expert_bias, "expert_bias", torch.float32, (cfg.E,), dev)
    ps = None if W_split is None else _need(W_split, "W_split", torch.bfloat16, (3, cfg.E, cfg.H), dev)
    if out is None:
        idx = torch.empty(cfg.T, cfg.k, dtype=torch.int32, device=dev)
        w = torch.empty(cfg.T, cfg.k, dtype=torch.float32, device=dev)
        counts = torch.empty(cfg.E, dtype=torch.int32, device=dev)
        aux_P = torch.empty(cfg.E, dtype=torch.float32, device=dev) if aux else None
        aux_loss = torch.empty(1, dtype=torch.float32, device=dev) if aux else None
    else:
        idx, w, counts, aux_P, aux_loss = out
    ws = _ws(ws, cfg, _lib.MOE_WS_ROUTE, dev)
    pP = None if aux_P is None else aux_P.data_ptr()
    pL = None if aux_loss is None else aux_loss.data_ptr()
    lib = _lib.load()
    if ps is None:
        rc = lib.moe_route(cfg.ref(), ph, pw, pb, idx.data_ptr(), w.data_ptr(), counts.data_ptr(),
                           pP, pL, ws.ptr, ws.nbytes, _stream(dev))
        _lib.check(rc, "moe_route")
    else:
        rc = lib.moe_route_prepared(cfg.ref(), ph, pw, ps, pb, idx.data_ptr(), w.data_ptr(),
                                    counts.data_ptr(), pP, pL, ws.ptr, ws.nbytes, _stream(dev))
        _lib.check(rc, "moe_route_prepared")
    return idx, w, counts, aux_P, aux_loss


def router_logits(cfg: MoeConfig, hidden, W_router, *, ws: Optional[Workspace] = None):
    """moe_router_logits: fp32 logits [T, E]."""
    dev = hidden.device
    ph = _need(hidden, "hidden", torch.bfloat16, (cfg.T, cfg.H), dev)
    pw = _need(W_router, "W_router", torch.float32, (cfg.E, cfg.H), dev)
    logits = torch.empty(cfg.T, cfg.E, dtype=torch.float32, device=dev)
    ws = _ws(ws, cfg, _lib.MOE_WS_ROUTE, dev)
    _lib.check(_lib.load().moe_router_logits(cfg.ref(), ph, pw, logits.data_ptr(), ws.ptr, ws.nbytes,
                                             _stream(dev)), "moe_router_logits")
    return logits


def router_scores(logits):
    """moe_router_scores: the routing kernels' fp32 sigmoid of every logit."""
    dev = logits.device
    if logits.dtype != torch.float32 or not logits.is_contiguous() or logits.device.type != "cuda":
        raise ValueError("logits: contiguous fp32 CUDA tensor expected")
    out = torch.empty_like(logits)
    _lib.check(_lib.load().moe_router_scores(logits.data_ptr(), out.data_ptr(), logits.numel(), _stream(dev)),
               "moe_router_scores")
    return out


def route_from_logits(cfg: MoeConfig, logits, expert_bias=None, *, aux: bool = False,
                      ws: Optional[Workspace] = None):
    """moe_route_from_logits: same outputs as route(), from fp32 logits."""
    dev = logits.device
    pl = _need(logits, "logits", torch.float32, (cfg.T, cfg.E), dev)
    pb = _opt(expert_bias, "expert_bias", torch.float32, (cfg.E,), dev)
    idx = torch.empty(cfg.T, cfg.k, dtype=torch.int32, device=dev)
    w = torch.empty(cfg.T, cfg.k, dtype=torch.float32, device=dev)
    counts = torch.empty(cfg.E, dtype=torch.int32, device=dev)
    aux_P = torch.empty(cfg.E, dtype=torch.float32, device=dev) if aux else None
    aux_loss = torch.empty(1, dtype=torch.float32, device=dev) if aux else None
    ws = _ws(ws, cfg, _lib.MOE_WS_ROUTE, dev)
    rc = _lib.load().moe_route_from_logits(cfg.ref(), pl, pb, idx.data_ptr(), w.data_ptr(),
                                           counts.data_ptr(), None if aux_P is None else aux_P.data_ptr(),
                                           None if aux_loss is None else aux_loss.data_ptr(), ws.ptr, ws.nbytes,
                                           _stream(dev))
    _lib.check(rc, "moe_route_from_logits")
    return idx, w, counts, aux_P, aux_loss


def forward(cfg: MoeConfig, hidden, W_gate_up, W_down, shared_gate_up, shared_down, topk_idx, topk_w,
            residual=None, *, ws: Optional[Workspace] = None, out=None):
    """moe_forward: out [T, H] bf16 = sum_j w * SwiGLU_e(x) + shared(x) (+ residual)."""
    dev = hidden.device
    bf = torch.bfloat16
    ph = _need(hidden, "hidden", bf, (cfg.T, cfg.H), dev)
    pgu = _need(W_gate_up, "W_gate_up", bf, (cfg.E, 2 * cfg.I, cfg.H), dev)
    pd = _need(W_down, "W_down", bf, (cfg.E, cfg.I, cfg.H), dev)
    psgu = _need(shared_gate_up, "shared_gate_up", bf, (2 * cfg.Is, cfg.H), dev)
    psd = _need(shared_down, "shared_down", bf, (cfg.Is, cfg.H), dev)
    pi = _need(topk_idx, "topk_idx", torch.int32, (cfg.T, cfg.k), dev)
    pw = _need(topk_w, "topk_w", torch.float32, (cfg.T, cfg.k), dev)
    pr = _opt(residual, "residual", bf, (cfg.T, cfg.H), dev)
    if out is None:
        out = torch.empty(cfg.T, cfg.H, dtype=bf, device=dev)
    po = _need(out, "out", bf, (cfg.T, cfg.H), dev)
    ws = _ws(ws, cfg, _lib.MOE_WS_FORWARD, dev)
    rc = _lib.load().moe_forward(cfg.ref(), ph, pgu, pd, psgu, psd, pi, pw, pr, po, ws.ptr, ws.nbytes,
                                 _stream(dev))
    _lib.check(rc, "moe_forward")
    return out


def layer(cfg: MoeConfig, hidden, W_router, expert_bias, W_gate_up, W_down, shared_gate_up, shared_down,
          residual=None, *, W_split=None, flags: int = 0, ws: Optional[Workspace] = None, out=None, routing=None,
          aux: bool = False):
    """moe_layer: routing and the expert stage in one call (with
    flags=MOE_LAYER_FUSED_ROUTER, the fused router where the shape allows it;
    with MOE_LAYER_FUSED_COMBINE, the combine in the shared expert's down
    GEMM; see include/moe.h).  Returns (out, (topk_idx, topk_w, expert_counts)),
    or with aux=True (out, (topk_idx, topk_w, expert_counts, aux_P [E],
    aux_loss [1])); `routing` (such a tuple) is filled instead of
    allocating."""
    dev = hidden.device
    bf = torch.bfloat16
    ph = _need(hidden, "hidden", bf, (cfg.T, cfg.H), dev)
    pwr = _need(W_router, "W_router", torch.float32, (cfg.E, cfg.H), dev)
    psp = _opt(W_split, "W_split", bf, (3, cfg.E, cfg.H), dev)
    pb = _opt(expert_bias, "expert_bias", torch.float32, (cfg.E,), dev)
    pgu = _need(W_gate_up, "W_gate_up", bf, (cfg.E, 2 * cfg.I, cfg.H), dev)
    pd = _need(W_down, "W_down", bf, (cfg.E, cfg.I, cfg.H), dev)
    psgu = _need(shared_gate_up, "shared_gate_up", bf, (2 * cfg.Is, cfg.H), dev)
    psd = _need(shared_down, "shared_down", bf, (cfg.Is, cfg.H), dev)
    pr = _opt(residual, "residual", bf, (cfg.T, cfg.H), dev)
    if routing is None or len(routing) != (5 if aux else 3):
        routing = (torch.empty(cfg.T, cfg.k, dtype=torch.int32, device=dev),
                   torch.empty(cfg.T, cfg.k, dtype=torch.float32, device=dev),
                   torch.empty(cfg.E, dtype=torch.int32, device=dev))
        if aux:
            routing += (torch.empty(cfg.E, dtype=torch.float32, device=dev),
                        torch.empty(1, dtype=torch.float32, device=dev))
    pi = _need(routing[0], "topk_idx", torch.int32, (cfg.T, cfg.k), dev)
    pw = _need(routing[1], "topk_w", torch.float32, (cfg.T, cfg.k), dev)
    pc = _need(routing[2], "expert_counts", torch.int32, (cfg.E,), dev)
    pP = _need(routing[3], "aux_P", torch.float32, (cfg.E,), dev) if aux else None
    pl = _need(routing[4], "aux_loss", torch.float32, (1,), dev) if aux else None
    if out is None:
        out = torch.empty(cfg.T, cfg.H, dtype=bf, device=dev)
    po = _need(out, "out", bf, (cfg.T, cfg.H), dev)
    if ws is None:
        ws = Workspace(cfg, WS_LAYER, dev, flags)
    elif ws.which != WS_LAYER or not ws.fits(cfg, flags):
        raise ValueError("workspace of the wrong kind or too small")
    rc = _lib.load().moe_layer(cfg.ref(), ph, pwr, psp, pb, pgu, pd, psgu, psd, pr, pi, pw, pc, pP, pl,
                               po, flags, ws.ptr, ws.nbytes, _stream(dev))
    _lib.check(rc, "moe_layer")
    return out, routing


def backward(cfg: MoeConfig, hidden, W_gate_up, W_down, shared_gate_up, shared_down, topk_idx, topk_w, d_out,
             *, ws: Optional[Workspace] = None, out: Optional[dict] = None):
    """moe_backward (routing fixed): dict(d_hidden [T,H] bf16, dW_gate_up
    [E,2I,H] fp32, dW_down [E,I,H] fp32, d_shared_gate_up [2Is,H] fp32,
    d_shared_down [Is,H] fp32, d_topk_w [T,k] fp32); `out` (a dict like the
    result) is filled instead of allocating."""
    dev = hidden.device
    bf = torch.bfloat16
    ph = _need(hidden, "hidden", bf, (cfg.T, cfg.H), dev)
    pgu = _need(W_gate_up, "W_gate_up", bf, (cfg.E, 2 * cfg.I, cfg.H), dev)
    pd = _need(W_down, "W_down", bf, (cfg.E, cfg.I, cfg.H), dev)
    psgu = _need(shared_gate_up, "shared_gate_up", bf, (2 * cfg.Is, cfg.H), dev)
    psd = _need(shared_down, "shared_down", bf, (cfg.Is, cfg.H), dev)
    pi = _need(topk_idx, "topk_idx", torch.int32, (cfg.T, cfg.k), dev)
    pw = _need(topk_w, "topk_w", torch.float32, (cfg.T, cfg.k), dev)
    pdo = _need(d_out, "d_out", bf, (cfg.T, cfg.H), dev)
    f32 = torch.float32
    shapes = dict(d_hidden=((cfg.T, cfg.H), bf), dW_gate_up=((cfg.E, 2 * cfg.I, cfg.H), f32),
                  dW_down=((cfg.E, cfg.I, cfg.H), f32), d_shared_gate_up=((2 * cfg.Is, cfg.H), f32),
                  d_shared_down=((cfg.Is, cfg.H), f32), d_topk_w=((cfg.T, cfg.k), f32))
    g = {}
    for name, (shape, dt) in shapes.items():
        t = out.get(name) if out else None
        if t is None:
            t = torch.empty(*shape, dtype=dt, device=dev)
        _need(t, name, dt, shape, dev)
        g[name] = t
    ws = _ws(ws, cfg, _lib.MOE_WS_BACKWARD, dev)
    rc = _lib.load().moe_backward(cfg.ref(), ph, pgu, pd, psgu, psd, pi, pw, pdo,
                                  g["d_hidden"].data_ptr(), g["dW_gate_up"].data_ptr(), g["dW_down"].data_ptr(),
                                  g["d_shared_gate_up"].data_ptr(), g["d_shared_down"].data_ptr(),
                                  g["d_topk_w"].data_ptr(), ws.ptr, ws.nbytes, _stream(dev))
    _lib.check(rc, "moe_backward")
    return g


class DenseWorkspace:
    """A device workspace for moe_dense_ffn (T tokens, hidden H, inner size I)."""

    def __init__(self, T: int, H: int, I: int, device=None):
        self.shape = (T, H, I)
        self.nbytes = int(_lib.load().moe_dense_workspace_bytes(T, H, I))
        if self.nbytes == 0:
            raise ValueError("unsupported dense shape T=%d H=%d I=%d" % (T, H, I))
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device or "cuda")
        assert self.buf.data_ptr() % 256 == 0
        _lib.check(_lib.load().moe_workspace_init(self.ptr, self.nbytes, _stream(self.buf.device)),
                   "moe_workspace_init")

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()

    def status(self, reset: bool = True) -> int:
        v = ctypes.c_int32(0)
        _lib.check(_lib.load().moe_get_status(self.ptr, self.nbytes, _stream(self.buf.device), ctypes.byref(v),
                                              1 if reset else 0), "moe_get_status")
        return int(v.value)


def dense_ffn(hidden, W_gate_up, W_down, residual=None, *, ws: Optional[DenseWorkspace] = None, out=None):
    """moe_dense_ffn: out [T, H] bf16 = down(silu(gate x) * up x) (+ residual),
    W_gate_up [2I, H] (gate rows, then up rows), W_down [I, H]."""
    dev = hidden.device
    bf = torch.bfloat16
    T, H = hidden.shape
    I = W_down.shape[0]
    ph = _need(hidden, "hidden", bf, (T, H), dev)
    pgu = _need(W_gate_up, "W_gate_up", bf, (2 * I, H), dev)
    pd = _need(W_down, "W_down", bf, (I, H), dev)
    pr = _opt(residual, "residual", bf, (T, H), dev)
    if out is None:
        out = torch.empty(T, H, dtype=bf, device=dev)
    po = _need(out, "out", bf, (T, H), dev)
    if ws is None or ws.shape != (T, H, I):
        ws = DenseWorkspace(T, H, I, dev)
    rc = _lib.load().moe_dense_ffn(T, H, I, ph, pgu, pd, pr, po, ws.ptr, ws.nbytes, _stream(dev))
    _lib.check(rc, "moe_dense_ffn")
    return out


class SizedWorkspace:
    """A device workspace of a given byte size (the expert-parallel calls)."""

    def __init__(self, nbytes: int, what: str, device=None):
        if nbytes == 0:
            raise ValueError("unsupported shape for %s" % what)
        self.nbytes = int(nbytes)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device or "cuda")
        assert self.buf.data_ptr() % 256 == 0
        _lib.check(_lib.load().moe_workspace_init(self.ptr, self.nbytes, _stream(self.buf.device)),
                   "moe_workspace_init")

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()

    def status(self, reset: bool = True) -> int:
        v = ctypes.c_int32(0)
        _lib.check(_lib.load().moe_get_status(self.ptr, self.nbytes, _stream(self.buf.device), ctypes.byref(v),
                                              1 if reset else 0), "moe_get_status")
        return int(v.value)


def ep_dispatch_workspace_bytes(cfg: MoeConfig, ranks: int) -> int:
    """moe_ep_dispatch_workspace_bytes (0: the shape is not supported)."""
    return int(_lib.load().moe_ep_dispatch_workspace_bytes(cfg.ref(), ranks))


def expert_rows_workspace_bytes(cfg: MoeConfig, rows: int) -> int:
    """moe_expert_rows_workspace_bytes (0: the shape is not supported)."""
    return int(_lib.load().moe_expert_rows_workspace_bytes(cfg.ref(), rows))


def ep_dispatch(cfg: MoeConfig, ranks: int, hidden, topk_idx, *, ws: Optional[SizedWorkspace] = None):
    """moe_ep_dispatch: the pairs grouped by the rank holding their expert.
    Returns (send_counts [ranks] int32, x_send [kT, H] bf16, e_send [kT] int32
    local expert ids, slot_of [T, k] int32)."""
    dev = hidden.device
    ph = _need(hidden, "hidden", torch.bfloat16, (cfg.T, cfg.H), dev)
    pi = _need(topk_idx, "topk_idx", torch.int32, (cfg.T, cfg.k), dev)
    n = cfg.T * cfg.k
    counts = torch.empty(ranks, dtype=torch.int32, device=dev)
    x_send = torch.empty(n, cfg.H, dtype=torch.bfloat16, device=dev)
    e_send = torch.empty(n, dtype=torch.int32, device=dev)
    slot_of = torch.empty(cfg.T, cfg.k, dtype=torch.int32, device=dev)
    need = int(_lib.load().moe_ep_dispatch_workspace_bytes(cfg.ref(), ranks))
    if need and (ws is None or ws.nbytes < need):
        ws = SizedWorkspace(need, "moe_ep_dispatch", dev)
    # (an unsupported shape has no workspace size: the call itself names the error)
    rc = _lib.load().moe_ep_dispatch(cfg.ref(), ranks, ph, pi, counts.data_ptr(), x_send.data_ptr(),
                                     e_send.data_ptr(), slot_of.data_ptr(), ws.ptr if need else None,
                                     ws.nbytes if need else 0, _stream(dev))
    _lib.check(rc, "moe_ep_dispatch")
    return counts, x_send, e_send, slot_of


def expert_rows(cfg: MoeConfig, x, expert, W_gate_up, W_down, *, ws: Optional[SizedWorkspace] = None, out=None):
    """moe_expert_rows: y[i] = expert[i]'s SwiGLU FFN of x[i] (unweighted), with
    cfg.E local experts' weights W_gate_up [E, 2I, H] / W_down [E, I, H]."""
    dev = x.device
    rows = x.shape[0]
    px = _need(x, "x", torch.bfloat16, (rows, cfg.H), dev)
    pe = _need(expert, "expert", torch.int32, (rows,), dev)
    pgu = _need(W_gate_up, "W_gate_up", torch.bfloat16, (cfg.E, 2 * cfg.I, cfg.H), dev)
    pd = _need(W_down, "W_down", torch.bfloat16, (cfg.E, cfg.I, cfg.H), dev)
    if out is None:
        out = torch.empty(rows, cfg.H, dtype=torch.bfloat16, device=dev)
    po = _need(out, "out", torch.bfloat16, (rows, cfg.H), dev)
    if rows == 0:
        return out
    need = int(_lib.load().moe_expert_rows_workspace_bytes(cfg.ref(), rows))
    if need and (ws is None or ws.nbytes < need):
        ws = SizedWorkspace(need, "moe_expert_rows", dev)
    rc = _lib.load().moe_expert_rows(cfg.ref(), rows, px, pe, pgu, pd, po, ws.ptr if need else None,
                                     ws.nbytes if need else 0, _stream(dev))
    _lib.check(rc, "moe_expert_rows")
    return out


def combine(cfg: MoeConfig, Y, shared_row0: int, slot_of, topk_w, residual=None, out=None):
    """moe_combine: out[t] = bf16(sum_j w[t,j] Y[slot_of[t,j]] + Y[shared_row0 + t] (+ residual[t]))."""
    dev = Y.device
    rows = Y.shape[0]
    py = _need(Y, "Y", torch.bfloat16, (rows, cfg.H), dev)
    ps = _need(slot_of, "slot_of", torch.int32, (cfg.T, cfg.k), dev)
    pw = _need(topk_w, "topk_w", torch.float32, (cfg.T, cfg.k), dev)
    pr = _opt(residual, "residual", torch.bfloat16, (cfg.T, cfg.H), dev)
    if out is None:
        out = torch.empty(cfg.T, cfg.H, dtype=torch.bfloat16, device=dev)
    po = _need(out, "out", torch.bfloat16, (cfg.T, cfg.H), dev)
    rc = _lib.load().moe_combine(cfg.ref(), py, rows, shared_row0, ps, pw, pr, po, _stream(dev))
    _lib.check(rc, "moe_combine")
    return out


def expert_feedback(cfg: MoeConfig, counts, gamma: float, expert_bias=None, totals=None) -> None:
    """moe_expert_feedback: in place, bias += +-gamma toward the balanced load
    (routing article §三) and totals += counts (§六)."""
    dev = counts.device
    pc = _need(counts, "expert_counts", torch.int32, (cfg.E,), dev)
    pb = _opt(expert_bias, "expert_bias", torch.float32, (cfg.E,), dev)
    pt = _opt(totals, "totals", torch.int64, (cfg.E,), dev)
    _lib.check(_lib.load().moe_expert_feedback(cfg.ref(), pc, gamma, pb, pt, _stream(dev)),
               "moe_expert_feedback")


def rmsnorm(x, eps: float = 1e-6, out=None):
    """moe_rmsnorm: bf16(x / sqrt(mean(x^2) + eps)) per row (decoder pre-norm)."""
    T, H = x.shape
    _need(x, "x", torch.bfloat16, (T, H), x.device)
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", torch.bfloat16, (T, H), x.device)
    _lib.check(_lib.load().moe_rmsnorm(T, H, x.data_ptr(), out.data_ptr(), eps, _stream(x.device)), "moe_rmsnorm")
    return out


def _sized(ws: Optional[SizedWorkspace], need: int, what: str, device) -> Optional[SizedWorkspace]:
    """ws, or one of `need` bytes where none was given.  One that is too small is
    refused: its owner would look for the call's status in it."""
    if ws is not None and ws.nbytes < need:
        raise ValueError("workspace too small for %s: %d bytes, needs %d" % (what, ws.nbytes, need))
    return SizedWorkspace(need, what, device) if ws is None and need else ws


def block_norm_workspace_bytes(T: int, H: int, groups: int = 1) -> int:
    """moe_block_norm_workspace_bytes (0: the shape is not supported).  Fewer groups
    may need more: each has its own plan."""
    return int(_lib.load().moe_block_norm_workspace_bytes(T, H, groups))


def block_norm_workspace(T: int, H: int, groups: int = 1, device=None) -> SizedWorkspace:
    """The workspace of block_norm_backward (groups: rows of its gate, 1 without)."""
    return SizedWorkspace(block_norm_workspace_bytes(T, H, groups), "moe_block_norm_backward", device)


def _block_norm_args(x, y, gate, w_post, w_pre):
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise TypeError("x must be a [T, H] tensor")
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("x must be torch.bfloat16 or torch.float32, got %s" % x.dtype)
    dev = x.device
    T, H = x.shape
    groups = 1 if gate is None else gate.shape[0]
    px = _need(x, "x", x.dtype, (T, H), dev)
    py = _opt(y, "y", torch.bfloat16, (T, H), dev)
    pg = _opt(gate, "gate", torch.float32, (groups, H), dev)
    pp = _opt(w_post, "w_post", torch.float32, (H,), dev)
    pq = _opt(w_pre, "w_pre", torch.float32, (H,), dev)
    return T, H, groups, int(x.dtype == torch.float32), px, py, pg, pp, pq


def block_norm(x, y=None, gate=None, w_post=None, w_pre=None, *, alpha: float = 1.0, eps: float = 1e-6, out=None):
    """moe_block_norm: (r, n) with r = alpha x + gate RMS(y) w_post (the new
    residual stream, x's type) and n = RMS(r) w_pre (the next block's input,
    bf16).  x [T, H] bf16 or fp32, y [T, H] bf16 (None: r = alpha x), gate
    [groups, H] fp32 with T % groups == 0, w_post and w_pre [H] fp32 (None: 1).
    `out` = (r, n) is filled instead of allocating; r may be x, n may be y."""
    T, H, groups, f32, px, py, pg, pp, pq = _block_norm_args(x, y, gate, w_post, w_pre)
    dev = x.device
    if out is None:
        r = torch.empty_like(x)
        n = torch.empty_like(x, dtype=torch.bfloat16) if f32 else torch.empty_like(x)
        pr, pn = r.data_ptr(), n.data_ptr()
    else:
        r, n = out
        pr = _need(r, "r", x.dtype, (T, H), dev)
        pn = _need(n, "n", torch.bfloat16, (T, H), dev)
    _lib.check(_lib.load().moe_block_norm(T, H, groups, f32, px, py, pg, pp, pq, alpha, eps, pr, pn, _stream(dev)),
               "moe_block_norm")
    return r, n


def block_norm_backward(x, y, gate, w_post, w_pre, d_r, d_n, *, alpha: float = 1.0, eps: float = 1e-6,
                        ws: Optional[SizedWorkspace] = None, out: Optional[dict] = None):
    """moe_block_norm_backward: the gradients of block_norm(x, y, gate, w_post,
    w_pre) from d_r [T, H] (x's type; None: zero) and d_n [T, H] bf16, as
    dict(d_x, d_y, d_gate [groups, H], dw_post [H], dw_pre [H]), the vectors in
    fp32; without y only d_x and dw_pre.  `out` (a dict like the result) is
    filled instead of allocating; its d_x may be d_r, its d_y may be d_n."""
    T, H, groups, f32, px, py, pg, pp, pq = _block_norm_args(x, y, gate, w_post, w_pre)
    dev = x.device
    pdr = _opt(d_r, "d_r", x.dtype, (T, H), dev)
    pdn = _need(d_n, "d_n", torch.bfloat16, (T, H), dev)
    vec = torch.float32
    shapes = dict(d_x=((T, H), x.dtype), dw_pre=((H,), vec))
    if y is not None:
        shapes.update(d_y=((T, H), torch.bfloat16), d_gate=((groups, H), vec), dw_post=((H,), vec))
    g = {}
    for name, (shape, dt) in shapes.items():
        t = out.get(name) if out else None
        if t is None:
            t = torch.empty(shape, dtype=dt, device=dev)
        else:
            _need(t, name, dt, shape, dev)
        g[name] = t
    need = int(_lib.load().moe_block_norm_workspace_bytes(T, H, groups))
    ws = _sized(ws, need, "moe_block_norm_backward", dev)
    # (an unsupported shape has no workspace size: the call itself names the error)
    ptr = {name: t.data_ptr() for name, t in g.items()}
    rc = _lib.load().moe_block_norm_backward(T, H, groups, f32, px, py, pg, pp, pq, alpha, eps, pdr, pdn, ptr["d_x"],
                                             ptr.get("d_y"), ptr.get("d_gate"), ptr.get("dw_post"), ptr["dw_pre"],
                                             ws.ptr if need else None, ws.nbytes if need else 0, _stream(dev))
    _lib.check(rc, "moe_block_norm_backward")
    return g


def vocab_loss_workspace(T: int, H: int, V: int, backward: bool = False, device=None) -> SizedWorkspace:
    """The workspace of vocab_loss, or with backward=True of vocab_loss_backward."""
    return SizedWorkspace(_lib.load().moe_vocab_loss_workspace_bytes(T, H, V, int(backward)), "moe_vocab_loss",
                          device)


def _vocab_args(hidden, W_vocab, target, backward, ws):
    for name, t in (("hidden", hidden), ("W_vocab", W_vocab)):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise TypeError("%s must be a 2-dimensional tensor" % name)
    dev = hidden.device
    T, H = hidden.shape
    V = W_vocab.shape[0]
    ph = _need(hidden, "hidden", torch.bfloat16, (T, H), dev)
    pw = _need(W_vocab, "W_vocab", torch.bfloat16, (V, H), dev)
    if not isinstance(target, torch.Tensor) or target.dtype not in (torch.int32, torch.int64):
        raise TypeError("target must be a torch.int32 or torch.int64 tensor")
    pt = _need(target, "target", target.dtype, (T,), dev)
    need = int(_lib.load().moe_vocab_loss_workspace_bytes(T, H, V, int(backward)))
    ws = _sized(ws, need, "moe_vocab_loss", dev)
    # (an unsupported shape has no workspace size: the call itself names the error;
    # the caller holds on to ws until the launches are enqueued)
    bits = 64 if target.dtype == torch.int64 else 32
    return (T, H, V, ph, pw, pt, bits), (ws.ptr if need else None, ws.nbytes if need else 0, _stream(dev)), ws


def vocab_loss(hidden, W_vocab, target, *, ignore_index: int = -100, ws: Optional[SizedWorkspace] = None, out=None):
    """moe_vocab_loss: (loss [T] fp32, lse [T] fp32) of the softmax cross entropy
    of hidden [T, H] bf16 over the vocabulary W_vocab [V, H] bf16; target [T]
    int32 or int64, rows with target == ignore_index give zeros.  No reduction:
    the mean is loss.sum() / (rows that count).  `out` = (loss, lse) is filled
    instead of allocating."""
    a, z, ws = _vocab_args(hidden, W_vocab, target, False, ws)
    T, dev = a[0], hidden.device
    loss, lse = out if out is not None else (torch.empty(T, dtype=torch.float32, device=dev) for _ in range(2))
    pl = _need(loss, "loss", torch.float32, (T,), dev)
    pe = _need(lse, "lse", torch.float32, (T,), dev)
    _lib.check(_lib.load().moe_vocab_loss(*a, ignore_index, pl, pe, *z), "moe_vocab_loss")
    return loss, lse


def vocab_loss_backward(hidden, W_vocab, target, lse, d_loss, *, ignore_index: int = -100,
                        ws: Optional[SizedWorkspace] = None, out: Optional[dict] = None):
    """moe_vocab_loss_backward: dict(d_hidden [T, H] bf16, dW_vocab [V, H] bf16)
    from d_loss [T] fp32 (1 / n on every row for the mean over n) and vocab_loss's
    lse; `out` (a dict like the result) is filled instead of allocating."""
    a, z, ws = _vocab_args(hidden, W_vocab, target, True, ws)
    T, dev = a[0], hidden.device
    pe = _need(lse, "lse", torch.float32, (T,), dev)
    pd = _need(d_loss, "d_loss", torch.float32, (T,), dev)
    g = {}
    for name, like in (("d_hidden", hidden), ("dW_vocab", W_vocab)):
        t = out.get(name) if out else None
        if t is None:
            t = torch.empty_like(like)
        _need(t, name, torch.bfloat16, like.shape, dev)
        g[name] = t
    _lib.check(_lib.load().moe_vocab_loss_backward(*a, ignore_index, pe, pd, g["d_hidden"].data_ptr(),
                                                   g["dW_vocab"].data_ptr(), *z), "moe_vocab_loss_backward")
    return g


def route_backward_workspace(cfg: MoeConfig, device=None) -> SizedWorkspace:
    """The workspace of route_backward."""
    return SizedWorkspace(_lib.load().moe_route_backward_workspace_bytes(cfg.ref()),
                          "moe_route_backward", device)


def route_backward(cfg: MoeConfig, hidden, W_router, topk_idx, d_topk_w, *, d_aux_loss=None, expert_counts=None,
                   d_hidden_add=None, W_split=None, ws: Optional[SizedWorkspace] = None, out: Optional[dict] = None):
    """moe_route_backward: the router's gradient for route()'s choice of experts,
    dict(d_hidden [T, H] bf16, dW_router [E, H] fp32), from d_topk_w [T, k]
    (backward()'s) and optionally d_aux_loss [1] with route()'s expert_counts;
    d_hidden_add [T, H] (backward()'s d_hidden) is added before the rounding.
    `out` (a dict like the result) is filled instead of allocating; its d_hidden
    may be d_hidden_add."""
    dev = hidden.device
    bf, f32 = torch.bfloat16, torch.float32
    ph = _need(hidden, "hidden", bf, (cfg.T, cfg.H), dev)
    pw = _need(W_router, "W_router", f32, (cfg.E, cfg.H), dev)
    ps = _opt(W_split, "W_split", bf, (3, cfg.E, cfg.H), dev)
    pi = _need(topk_idx, "topk_idx", torch.int32, (cfg.T, cfg.k), dev)
    pd = _need(d_topk_w, "d_topk_w", f32, (cfg.T, cfg.k), dev)
    pc = _opt(expert_counts, "expert_counts", torch.int32, (cfg.E,), dev)
    pa = _opt(d_aux_loss, "d_aux_loss", f32, (1,), dev)
    pp = _opt(d_hidden_add, "d_hidden_add", bf, (cfg.T, cfg.H), dev)
    g = {}
    for name, shape, dt in (("d_hidden", (cfg.T, cfg.H), bf), ("dW_router", (cfg.E, cfg.H), f32)):
        t = out.get(name) if out else None
        if t is None:
            t = torch.empty(*shape, dtype=dt, device=dev)
        _need(t, name, dt, shape, dev)
        g[name] = t
    need = int(_lib.load().moe_route_backward_workspace_bytes(cfg.ref()))
    ws = _sized(ws, need, "moe_route_backward", dev)
    rc = _lib.load().moe_route_backward(cfg.ref(), ph, pw, ps, pi, pd, pc, pa, pp,
                                        g["d_hidden"].data_ptr(), g["dW_router"].data_ptr(),
                                        ws.ptr if need else None, ws.nbytes if need else 0, _stream(dev))
    _lib.check(rc, "moe_route_backward")
    return g


# (without the checks around it, where torch has that call)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on(device, call, *args) -> int:
    """call(*args, the stream) with `device` the current one (its kernels and tensor
    maps are made there)."""
    if device.type != "cuda":
        raise ValueError("tensors on a CUDA device expected, got %s" % device)
    if device.index == _current_device():
        return call(*args, _stream(device))
    with torch.cuda.device(device):
        return call(*args, _stream(device))


@functools.lru_cache(maxsize=1024)
def _sort_tokens_bytes(T: int, k: int, E: int) -> int:
    return int(_lib.load().moe_sort_tokens_workspace_bytes(T, k, E))


def sort_tokens_workspace(T: int, k: int, E: int, device=None) -> SizedWorkspace:
    """The workspace of sort_tokens for T tokens with k experts each."""
    return SizedWorkspace(_sort_tokens_bytes(T, k, E), "moe_sort_tokens", device)


def sort_tokens(topk_idx, E: int, *, ws: Optional[SizedWorkspace] = None, out=None):
    """moe_sort_tokens: (offsets [E + 1] int32, slot_of [T, k] int32), the rows of a
    stable sort of the (token, j) pairs of topk_idx [T, k] int32 by expert: expert
    e has rows offsets[e] to offsets[e + 1] - 1, pair (t, j) row slot_of[t, j] (-1
    where topk_idx is -1: dropped).  `out` = (offsets, slot_of) is filled instead of
    allocating.  Ids that name no expert are dropped and noted in the workspace's
    status, which only a `ws` that is given lets its caller read."""
    T, k = _matrix(topk_idx, "topk_idx")
    dev = topk_idx.device
    i32 = torch.int32
    pi = _need(topk_idx, "topk_idx", i32, (T, k), dev)
    if out is None:
        offsets, slot_of = torch.empty(max(E, 0) + 1, dtype=i32, device=dev), torch.empty_like(topk_idx)
        po, ps = offsets.data_ptr(), slot_of.data_ptr()
    else:
        offsets, slot_of = out
        po = _need(offsets, "offsets", i32, (E + 1,), dev)
        ps = _need(slot_of, "slot_of", i32, (T, k), dev)
    need = _sort_tokens_bytes(T, k, E)
    ws = _sized(ws, need, "moe_sort_tokens", dev)
    # (an unsupported shape has no workspace size: the call itself names the error)
    _lib.check(_on(dev, _lib.load().moe_sort_tokens, T, k, E, pi, po, ps, ws.ptr if need else None,
                   ws.nbytes if need else 0), "moe_sort_tokens")
    return offsets, slot_of


def _slots(slot_of, dev):
    T, k = _matrix(slot_of, "slot_of")
    return T, k, _need(slot_of, "slot_of", torch.int32, (T, k), dev)


def _matrix(t, name):
    shape = t.shape if isinstance(t, torch.Tensor) else ()
    if len(shape) != 2:
        raise TypeError("%s must be a 2-dimensional tensor" % name)
    return shape


def _row_type(t, name) -> int:
    if t.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("%s must be torch.bfloat16 or torch.float32, got %s" % (name, t.dtype))
    return int(t.dtype == torch.float32)


def sort_rows(x, slot_of, *, out=None):
    """moe_sort_rows: the rows of x [T, H] in the order of sort_tokens, out[slot_of[t,
    j]] = x[t], [T k, H] of x's type (any type of whole 16-byte rows).  `out` [rows,
    H] is filled instead of allocating; rows behind the last expert's stay as they
    were."""
    _, H = _matrix(x, "x")
    dev = x.device
    T, k, ps = _slots(slot_of, dev)
    px = _need(x, "x", x.dtype, (T, H), dev)
    if out is None:
        rows = T * k
        out = torch.empty(rows, H, dtype=x.dtype, device=dev)
        po = out.data_ptr()
    else:
        rows = _matrix(out, "out")[0]
        po = _need(out, "out", x.dtype, (rows, H), dev)
    _lib.check(_on(dev, _lib.load().moe_sort_rows, T, k, H * x.element_size(), rows, px, ps, po), "moe_sort_rows")
    return out


def unsort_rows(y, slot_of, topk_w=None, *, out=None):
    """moe_unsort_rows: out [T, H] = sum_j topk_w[t, j] y[slot_of[t, j]] of y [rows,
    H] (bf16 or fp32) and topk_w [T, k] fp32 (None: weights of 1)."""
    rows, H = _matrix(y, "y")
    f32 = _row_type(y, "y")
    dev = y.device
    T, k, ps = _slots(slot_of, dev)
    py = _need(y, "y", y.dtype, (rows, H), dev)
    pw = _opt(topk_w, "topk_w", torch.float32, (T, k), dev)
    if out is None:
        out = torch.empty(T, H, dtype=y.dtype, device=dev)
        po = out.data_ptr()
    else:
        po = _need(out, "out", y.dtype, (T, H), dev)
    _lib.check(_on(dev, _lib.load().moe_unsort_rows, T, k, H, f32, rows, py, ps, pw, po), "moe_unsort_rows")
    return out


def sort_rows_backward(d_rows, slot_of, *, out=None):
    """The gradient of sort_rows: d_x[t] = sum_j d_rows[slot_of[t, j]] (moe_unsort_rows
    with weights of 1)."""
    return unsort_rows(d_rows, slot_of, None, out=out)


def unsort_rows_backward(d_out, y, slot_of, topk_w, *, out: Optional[dict] = None):
    """moe_unsort_rows_backward: the gradients of unsort_rows(y, slot_of, topk_w) from
    d_out [T, H], as dict(d_y [rows, H], d_w [T, k] fp32).  `out` (a dict like the
    result) is filled instead of allocating; its d_y may be y, and rows of d_y
    behind the last expert's stay as they were."""
    rows, H = _matrix(y, "y")
    f32 = _row_type(y, "y")
    dev = y.device
    T, k, ps = _slots(slot_of, dev)
    py = _need(y, "y", y.dtype, (rows, H), dev)
    pd = _need(d_out, "d_out", y.dtype, (T, H), dev)
    pw = _need(topk_w, "topk_w", torch.float32, (T, k), dev)
    d_y, d_w = (out.get("d_y"), out.get("d_w")) if out else (None, None)
    if d_y is None:
        d_y = torch.empty_like(y)
        pdy = d_y.data_ptr()
    else:
        pdy = _need(d_y, "d_y", y.dtype, (rows, H), dev)
    if d_w is None:
        d_w = torch.empty_like(topk_w)
        pdw = d_w.data_ptr()
    else:
        pdw = _need(d_w, "d_w", torch.float32, (T, k), dev)
    _lib.check(_on(dev, _lib.load().moe_unsort_rows_backward, T, k, H, f32, rows, pd, py, ps, pw, pdy, pdw),
               "moe_unsort_rows_backward")
    return dict(d_y=d_y, d_w=d_w)


def last_launch_count() -> int:
    """Kernels the last call on this thread enqueued."""
    return int(_lib.load().moe_last_launch_count())


def profile_enable(on: bool = True, stages: bool = False) -> None:
    """Bracket every kernel the library launches with CUDA events, or with
    stages=True time the routing and bucketing kernels of a call as one
    interval ("router_plus_permute") and every other kernel on its own."""
    _lib.check(_lib.load().moe_profile_enable((2 if stages else 1) if on else 0), "moe_profile_enable")


def profile_read(reset: bool = True, expert_ops: bool = False) -> dict:
    """{kernel name: (total ms, launches)} recorded since the last reset, of the
    layer's and the training operators' kernels, or with expert_ops=True of those
    of token order, 8-bit products and the AdamW step."""
    lib = _lib.load()
    out = {}
    first = _lib.MOE_KERNEL_TRAIN_FIRST
    ids = [*range(_lib.MOE_KERNEL_COUNT), *range(first, first + _lib.MOE_KERNEL_TRAIN_COUNT)]
    if expert_ops:
        ids = range(_lib.MOE_KERNEL_OPS_FIRST, _lib.MOE_KERNEL_OPS_FIRST + _lib.MOE_KERNEL_OPS_COUNT)
    for kid in ids:
        ms = ctypes.c_double(0.0)
        n = ctypes.c_int32(0)
        _lib.check(lib.moe_profile_read(kid, ctypes.byref(ms), ctypes.byref(n), 1 if reset else 0),
                   "moe_profile_read")
        out[lib.moe_kernel_name(kid).decode()] = (float(ms.value), int(n.value))
    return out


class MoELayer:
    """One MoE layer: weights on the device plus its workspace(s).

    __call__(hidden) runs the one moe_layer call on the current stream (with
    `flags`: the fused router where it applies), or, with single_call=False,
    moe_route then moe_forward (the two calls of the C ABI; same outputs).
    aux=True also returns the balance loss (not with the fused router).  The
    router weight is split once at construction (prepare_router); call
    prepare() again after changing W_router in place.  Layers of a stack may
    share one workspace (ws_layer, or ws_route / ws_fwd for the two calls).

    `routing` is the last call's; calls write it to the same tensors each time,
    or to those given to the call (new_routing()), which no other call touches."""

    def __init__(self, cfg: MoeConfig, W_router, expert_bias, W_gate_up, W_down, shared_gate_up, shared_down,
                 aux: bool = False, ws_route: Optional[Workspace] = None, ws_fwd: Optional[Workspace] = None,
                 single_call: bool = True, flags: int = 0, ws_layer: Optional[Workspace] = None):
        if single_call and aux and (flags & _lib.MOE_LAYER_FUSED_ROUTER):
            raise ValueError("the fused router does not compute the balance loss")
        self.cfg = cfg
        self.W_router, self.expert_bias = W_router, expert_bias
        self.W_gate_up, self.W_down = W_gate_up, W_down
        self.shared_gate_up, self.shared_down = shared_gate_up, shared_down
        self.aux = aux
        self.single_call, self.flags = single_call, flags
        self.device = W_router.device
        if single_call:
            if ws_layer is not None and (ws_layer.which != WS_LAYER or not ws_layer.fits(cfg, flags)):
                raise ValueError("workspace of the wrong kind or too small")
            self.ws_layer = ws_layer or Workspace(cfg, WS_LAYER, self.device, flags)
            self.ws_route = self.ws_fwd = None
        else:
            self.ws_layer = None
            self.ws_route = ws_route or Workspace(cfg, _lib.MOE_WS_ROUTE, self.device)
            self.ws_fwd = ws_fwd or Workspace(cfg, _lib.MOE_WS_FORWARD, self.device)
        self.routing = None
        self._own_routing = None        # (kept: a captured call holds their addresses)
        self.last_launches = 0
        self.W_split = None
        self.prepare()

    def prepare(self) -> None:
        """(Re)make the bf16 x 3 split of W_router that routing reads."""
        self.W_split = prepare_router(self.cfg, self.W_router, out=self.W_split)

    def new_routing(self):
        """Tensors for one call's routing: (topk_idx, topk_w, expert_counts), with
        aux (.., aux_P, aux_loss)."""
        cfg, dev = self.cfg, self.device
        f32, i32 = torch.float32, torch.int32
        r = (torch.empty(cfg.T, cfg.k, dtype=i32, device=dev), torch.empty(cfg.T, cfg.k, dtype=f32, device=dev),
             torch.empty(cfg.E, dtype=i32, device=dev))
        if self.aux:
            return r + (torch.empty(cfg.E, dtype=f32, device=dev), torch.empty(1, dtype=f32, device=dev))
        return r if self.single_call else r + (None, None)

    def __call__(self, hidden, residual=None, out=None, routing=None):
        if routing is None:
            if self._own_routing is None or len(self._own_routing) != (5 if self.aux or not self.single_call else 3):
                self._own_routing = self.new_routing()
            routing = self._own_routing
        self._hidden = hidden
        if self.single_call:
            y, self.routing = layer(self.cfg, hidden, self.W_router, self.expert_bias, self.W_gate_up, self.W_down,
                                    self.shared_gate_up, self.shared_down, residual, W_split=self.W_split,
                                    flags=self.flags, ws=self.ws_layer, out=out, routing=routing, aux=self.aux)
            self.last_launches = last_launch_count()
            return y
        self.routing = route(self.cfg, hidden, self.W_router, self.expert_bias, aux=self.aux, ws=self.ws_route,
                             out=routing, W_split=self.W_split)
        n = last_launch_count()
        idx, w = routing[0], routing[1]
        y = forward(self.cfg, hidden, self.W_gate_up, self.W_down, self.shared_gate_up, self.shared_down, idx,
                    w, residual, ws=self.ws_fwd, out=out)
        self.last_launches = n + last_launch_count()
        return y

    def status(self) -> int:
        if self.single_call:
            st = self.ws_layer.status()
        else:
            st = self.ws_route.status() | self.ws_fwd.status()
        if getattr(self, "ws_bwd", None) is not None:
            st |= self.ws_bwd.status()
        return st

    def backward(self, d_out, out: Optional[dict] = None, call=None) -> dict:
        """Gradients of the last call's output w.r.t. its input, the expert
        weights and the routing weights, for that call's routing (moe_backward;
        the router's own gradient and the residual path are not included), or of
        an earlier call: `call` = (its hidden, the routing tensors it was given)."""
        if call is None and self.routing is None:
            raise RuntimeError("backward() needs a forward call first")
        hidden, routing = (self._hidden, self.routing) if call is None else call
        if getattr(self, "ws_bwd", None) is None:
            self.ws_bwd = Workspace(self.cfg, _lib.MOE_WS_BACKWARD, self.device)
        g = backward(self.cfg, hidden, self.W_gate_up, self.W_down, self.shared_gate_up, self.shared_down,
                     routing[0], routing[1], d_out, ws=self.ws_bwd, out=out)
        self.last_launches = last_launch_count()
        return g

    def feedback(self, gamma: float, totals=None) -> None:
        """After a call: nudge expert_bias toward balanced load from this
        step's expert counts and add them to `totals` (see expert_feedback)."""
        if self.routing is None:
            raise RuntimeError("feedback() needs a routed step first")
        if self.expert_bias is None:
            self.expert_bias = torch.zeros(self.cfg.E, dtype=torch.float32, device=self.W_router.device)
        expert_feedback(self.cfg, self.routing[2], gamma, self.expert_bias, totals)


class DenseLayer:
    """The dense first decoder layer (an ordinary SwiGLU MLP, routing article
    §五 "first_k_dense_replace = 1"): weights [2I, H] / [I, H] and a
    workspace; __call__(hidden, residual=None, out=None) runs moe_dense_ffn."""

    def __init__(self, W_gate_up, W_down, T: int):
        self.W_gate_up, self.W_down = W_gate_up, W_down
        self.device = W_down.device
        I, H = W_down.shape
        self.cfg = types.SimpleNamespace(T=T, H=H, I=I)
        self.ws = DenseWorkspace(T, H, I, self.device)
        self.last_launches = 0

    def __call__(self, hidden, residual=None, out=None):
        y = dense_ffn(hidden, self.W_gate_up, self.W_down, residual, ws=self.ws, out=out)
        self.last_launches = last_launch_count()
        return y

    def status(self) -> int:
        return self.ws.status()


class MoEStack:
    """Decoder-style stack of MoE layers (the routing article's layout after
    its dense first layer): x <- x + layer(rmsnorm(x)) for every layer, all
    layers sharing one pair of workspaces.  __call__(hidden, out=None) runs the
    whole stack on the current stream."""

    def __init__(self, layers, eps: float = 1e-6):
        self.layers = list(layers)
        self.cfg = self.layers[0].cfg
        self.device = self.layers[0].device
        self.eps = eps
        T, H = self.cfg.T, self.cfg.H
        self._x = [torch.empty(T, H, dtype=torch.bfloat16, device=self.device) for _ in range(2)]
        self._norm = torch.empty(T, H, dtype=torch.bfloat16, device=self.device)
        self.last_launches = 0

    def __call__(self, hidden, out=None):
        n = 0
        x = hidden
        for i, layer in enumerate(self.layers):
            rmsnorm(x, self.eps, out=self._norm)
            dst = out if (out is not None and i == len(self.layers) - 1) else self._x[i % 2]
            layer(self._norm, residual=x, out=dst)
            n += 1 + layer.last_launches
            x = dst
        self.last_launches = n
        return x

    def status(self) -> int:
        st = 0
        for L in self.layers:
            st |= L.status()
        return st


class GraphedStep:
    """One step of a MoELayer or MoEStack captured into a CUDA graph.

    The step's kernels (and their programmatic launch edges) are recorded once
    on static input/output buffers; __call__(hidden) copies the batch into the
    static input, replays the graph on the current stream and returns the
    static output (overwritten by the next call).  Replays skip the host side
    of every call (argument checks, tensor-map encoding, launches), which is
    most of the cost of a decode-sized step."""

    def __init__(self, model, example):
        dev = example.device
        self.model = model
        self.x = torch.empty_like(example)
        self.x.copy_(example)
        self.out = torch.empty_like(example)
        side = torch.cuda.Stream(dev)
        side.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(side):
            for _ in range(2):                  # first calls configure kernels and buffers
                model(self.x, out=self.out)
        torch.cuda.current_stream(dev).wait_stream(side)
        torch.cuda.synchronize(dev)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            model(self.x, out=self.out)
        self.last_launches = model.last_launches

    def replay(self):
        """Run the captured step on whatever the static input holds."""
        self.graph.replay()
        return self.out

    def __call__(self, hidden):
        self.x.copy_(hidden, non_blocking=True)
        return self.replay()

    def status(self) -> int:
        return self.model.status()


class HostPipeline:
    """Runs a MoELayer (or MoEStack) over batches that live in (pinned) host memory.

    Every batch is copied host -> device, run through the layer, and its
    output copied device -> host.  The copies run on their own streams with two
    device buffers per direction, so the upload of batch i+1 and the download
    of batch i-1 overlap the layer's kernels on batch i; the layer itself runs
    on the caller's current stream, one batch after the other."""

    def __init__(self, layer, depth: int = 2):
        cfg = layer.cfg
        dev = layer.device
        self.layer = layer
        self.depth = depth
        self.x_dev = [torch.empty(cfg.T, cfg.H, dtype=torch.bfloat16, device=dev) for _ in range(depth)]
        self.y_dev = [torch.empty(cfg.T, cfg.H, dtype=torch.bfloat16, device=dev) for _ in range(depth)]
        self.s_in = torch.cuda.Stream(dev)
        self.s_out = torch.cuda.Stream(dev)
        self.ev_loaded = [torch.cuda.Event() for _ in range(depth)]
        self.ev_done = [torch.cuda.Event() for _ in range(depth)]
        self.ev_saved = [torch.cuda.Event() for _ in range(depth)]
        self.launches = 0

    def run(self, host_in, host_out) -> None:
        """host_in[i] -> layer -> host_out[i] for every i (pinned bf16 [T, H])."""
        comp = torch.cuda.current_stream(self.x_dev[0].device)
        used = [False] * self.depth
        for i, (hi, ho) in enumerate(zip(host_in, host_out)):
            b = i % self.depth
            with torch.cuda.stream(self.s_in):
                if used[b]:
                    self.s_in.wait_event(self.ev_done[b])       # the layer has read this buffer
                self.x_dev[b].copy_(hi, non_blocking=True)
                self.ev_loaded[b].record(self.s_in)
            comp.wait_event(self.ev_loaded[b])
            if used[b]:
                comp.wait_event(self.ev_saved[b])               # the previous output has left
            self.layer(self.x_dev[b], out=self.y_dev[b])
            self.launches += self.layer.last_launches
            self.ev_done[b].record(comp)
            with torch.cuda.stream(self.s_out):
                self.s_out.wait_event(self.ev_done[b])
                ho.copy_(self.y_dev[b], non_blocking=True)
                self.ev_saved[b].record(self.s_out)
            used[b] = True
        for b in range(self.depth):
            if used[b]:
                comp.wait_event(self.ev_saved[b])               # the caller's stream sees every output
