"""Matrix products of 8-bit operands with a scale for each block of 128.

    x8 = quantize(x)                        # [T, K] bf16 or fp32 -> e4m3 with scales
    y = product(x8, W8)                     # [T, N] bf16 = x W^T, W8 = quantize(W [N, K])

for experts, with the rows sorted by expert (moe.sort_tokens):

    x8 = quantize(x, slot_of=slot_of)       # each token's row quantized once, written to its slots
    y = product(x8, W8, offsets=offsets)    # W8 = quantize(W [E, N, K])

and the gradients, from d_y [rows, N]:

    dy8, dy8_t = quantize_both(d_y, offsets=offsets)
    x8_t = quantize_columns(x, offsets=offsets)          # x [rows, K]
    d_x = product(dy8, W8_t, offsets=offsets)            # W8_t = quantize_columns(W)
    dW = weight_gradient(dy8_t, x8_t)                    # [E, N, K] fp32

An operand is a Scaled: values [.., R, K] in torch.float8_e4m3fn (or e5m2) and
scales [.., ceil(K / 128), R rounded up to 16] in torch.float8_e8m0fnu, a power of
two for each row and 128 along K.  quantize_columns gives the form of the
transpose, with a scale for each 128 rows; grouped rows start each group on a
multiple of 128 there, and `starts` counts the blocks of 128 before each group.
The kernels run in libglr_moe.so (include/moe.h)."""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib
from .moe import SizedWorkspace, _need, _on, _opt, _row_type, _sized, _slots

E4M3, E5M2, SCALE = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu
_FORMAT = {E4M3: 0, E5M2: 1}


class Scaled(NamedTuple):
    """An operand: values, scales and, for grouped columns, starts [E + 1] int32."""
    values: torch.Tensor
    scales: torch.Tensor
    starts: Optional[torch.Tensor] = None

    def dequantize(self) -> torch.Tensor:
        """The values they stand for, in fp32 (for inspection)."""
        K = self.values.shape[-1]
        R = self.values.shape[-2]
        s = self.scales.float()[..., :R].mT.repeat_interleave(128, dim=-1)[..., :K]
        return self.values.float() * s


def workspace(device=None) -> SizedWorkspace:
    """The workspace of product and weight_gradient: their status word (a time-out), which
    without a workspace of the caller's goes with a temporary one."""
    return SizedWorkspace(_lib.MOE_SCALED_WS_BYTES, "moe_scaled_product", device)


def _up(n: int, to: int) -> int:
    return -(-n // to) * to


def _format(dtype) -> int:
    if dtype not in _FORMAT:
        raise TypeError("dtype must be torch.float8_e4m3fn or torch.float8_e5m2, got %s" % (dtype,))
    return _FORMAT[dtype]


def _operand(shape, R, K, dtype, dev, out, name):
    """(Scaled, pointers) of an operand [*shape, R, K], made or given."""
    wv, wsc = (*shape, R, K), (*shape, -(-K // 128), (R + 15) & -16)
    if out is None:
        v, s = torch.empty(wv, dtype=dtype, device=dev), torch.empty(wsc, dtype=SCALE, device=dev)
        return Scaled(v, s), v.data_ptr(), s.data_ptr()
    return out, _need(out[0], name + ".values", dtype, wv, dev), _need(out[1], name + ".scales", SCALE, wsc, dev)


def _quantize(x, offsets, dtype, rows, columns, out, out_t):
    whole = x.shape if isinstance(x, torch.Tensor) else ()
    if len(whole) not in (2, 3):
        raise TypeError("x must be a [R, K] or [batch, R, K] tensor")
    f32, fmt = _row_type(x, "x"), _format(dtype)
    dev = x.device
    shape = whole[:-2]
    R, K = whole[-2:]
    batch = shape[0] if shape else 1
    px = _need(x, "x", x.dtype, whole, dev)
    E, po, starts, P = 0, None, None, _up(R, 16)
    if offsets is not None:
        if x.dim() != 2:
            raise ValueError("offsets go with x [R, K]")
        if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 2:
            raise TypeError("offsets must be a [E + 1] tensor")
        E = offsets.shape[0] - 1
        po = _need(offsets, "offsets", torch.int32, (E + 1,), dev)
        P = (R // 128 + E) * 128
        starts = torch.empty_like(offsets) if out_t is None else out_t[2]
    pq = ps = pt = pst = None
    if rows:
        out, pq, ps = _operand(shape, R, K, dtype, dev, out, "out")
    if columns:
        out_t, pt, pst = _operand(shape, K, P, dtype, dev, out_t, "out")
    pstart = _opt(starts, "starts", torch.int32, (E + 1,), dev) if E else None
    if R == 0 and E:
        starts.zero_()
    if batch and R:
        _lib.check(_on(dev, _lib.load().moe_scaled_quantize, batch, R, K, f32, fmt, px, pq, ps, pt, pst, E, po, pstart,
                       P), "moe_scaled_quantize")
    return out, None if out_t is None else Scaled(out_t[0], out_t[1], starts)


def quantize(x, *, slot_of=None, dtype=E4M3, out=None) -> Scaled:
    """moe_scaled_quantize: x [R, K] or [batch, R, K] (bf16 or fp32, K % 16 == 0) in
    the 8-bit format with a scale for each 128 of K.  With slot_of [R, k] (x [R, K],
    from moe.sort_tokens) each row is written to its slots: [R k, K]
    (moe_scaled_quantize_rows).  `out` (a Scaled) is filled instead of allocating;
    with slot_of it may have more or fewer rows, and those that no slot names stay as
    they were."""
    if slot_of is None:
        return _quantize(x, None, dtype, True, False, out, None)[0]
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise TypeError("x must be a [T, K] tensor")
    f32, fmt = _row_type(x, "x"), _format(dtype)
    dev = x.device
    T, k, psl = _slots(slot_of, dev)
    K = x.shape[1]
    px = _need(x, "x", x.dtype, (T, K), dev)
    rows = T * k if out is None else out[0].shape[0]
    out, pq, ps = _operand((), rows, K, dtype, dev, out, "out")
    _lib.check(_on(dev, _lib.load().moe_scaled_quantize_rows, T, k, K, f32, fmt, rows, px, psl, pq, ps),
               "moe_scaled_quantize_rows")
    return out


def quantize_columns(x, *, offsets=None, dtype=E4M3, out=None) -> Scaled:
    """moe_scaled_quantize of x's transpose: values [.., K, P] with a scale for each
    128 of x's rows, P = R rounded up to 16.  With offsets [E + 1] int32 (the rows of
    x grouped, as by moe.sort_tokens) P = 128 (R // 128 + E) and `starts` is set;
    what lies behind the last group's blocks is not written."""
    return _quantize(x, offsets, dtype, False, True, None, out)[1]


def quantize_both(x, *, offsets=None, dtype=E4M3, out=None):
    """(quantize(x), quantize_columns(x, offsets=offsets)) from one read of x; with
    offsets, rows of no group are left out of both.  `out`: a pair of Scaled."""
    a, b = out if out is not None else (None, None)
    return _quantize(x, offsets, dtype, True, True, a, b)


def _checked(t, name, dims):
    """(format, pointer of the values, of the scales) of an operand with its scales."""
    try:
        v, s = t[0], t[1]
        shape, fmt = v.shape, _FORMAT[v.dtype]
        R, K = shape[-2:]
        if (len(shape) == dims and s.dtype is SCALE and s.shape == (*shape[:-2], -(-K // 128), (R + 15) & -16) and
                v.is_contiguous() and s.is_contiguous() and v.get_device() == s.get_device()):
            return fmt, v.data_ptr(), s.data_ptr()
    except (TypeError, KeyError, IndexError, ValueError, AttributeError):
        pass
    # what is wrong with it
    if not isinstance(t, tuple) or len(t) < 2 or not all(isinstance(v, torch.Tensor) for v in t[:2]):
        raise TypeError("%s must be a Scaled" % name)
    v, s = t[0], t[1]
    fmt = _format(v.dtype)
    if v.dim() != dims:
        raise ValueError("%s.values must have %d dimensions, got shape %s" % (name, dims, tuple(v.shape)))
    R, K = v.shape[-2:]
    return (fmt, _need(v, name + ".values", v.dtype, tuple(v.shape), v.device),
            _need(s, name + ".scales", SCALE, (*v.shape[:-2], -(-K // 128), _up(R, 16)), v.device))


def _result(out, dtype, shape, dev):
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("dtype must be torch.bfloat16 or torch.float32, got %s" % (dtype,))
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
        return out, out.data_ptr(), int(dtype == torch.float32)
    return out, _need(out, "out", dtype, shape, dev), int(dtype == torch.float32)


def product(a: Scaled, b: Scaled, *, offsets=None, dtype=torch.bfloat16, ws: Optional[SizedWorkspace] = None, out=None):
    """moe_scaled_product: a b^T, [M, N] in bf16 or fp32 (`dtype`), of a [M, K] and b
    [N, K].  With offsets [E + 1] int32 the rows of a are grouped and b is [E, N, K];
    rows of `out` that belong to no group stay as they were."""
    fa, pa, psa = _checked(a, "a", 2)
    fb, pb, psb = _checked(b, "b", 2 if offsets is None else 3)
    dev = a[0].device
    M, K = a[0].shape
    N, Kb = b[0].shape[-2:]
    if Kb != K or b[0].device != dev:
        raise ValueError("b's rows must be of a's length %d on %s, got %d on %s" % (K, dev, Kb, b[0].device))
    E, po = 0, None
    if offsets is not None:
        E = b[0].shape[0]
        po = _need(offsets, "offsets", torch.int32, (E + 1,), dev)
    out, pout, f32 = _result(out, dtype, (M, N), dev)
    ws = _sized(ws, _lib.MOE_SCALED_WS_BYTES, "moe_scaled_product", dev)
    _lib.check(_on(dev, _lib.load().moe_scaled_product, M, N, K, E, fa, fb, f32, pa, psa, pb, psb, po, pout, ws.ptr,
                   ws.nbytes), "moe_scaled_product")
    return out


def weight_gradient(dy_t: Scaled, x_t: Scaled, *, dtype=torch.float32, ws: Optional[SizedWorkspace] = None, out=None):
    """moe_scaled_weight_gradient: d_y^T x of quantize_columns(d_y) [N, P] and
    quantize_columns(x) [K, P]: [N, K], or with grouped columns (both of the same
    offsets, which is not looked at) [E, N, K], zeros for a group without rows."""
    fa, pa, psa = _checked(dy_t, "dy_t", 2)
    fb, pb, psb = _checked(x_t, "x_t", 2)
    dev = dy_t[0].device
    N, P = dy_t[0].shape
    K = x_t[0].shape[0]
    starts = dy_t[2] if len(dy_t) > 2 else None
    if x_t[0].shape[1] != P or x_t[0].device != dev:
        raise ValueError("x_t's rows must be of dy_t's length %d on %s, got %d on %s" %
                         (P, dev, x_t[0].shape[1], x_t[0].device))
    if (starts is None) != (len(x_t) < 3 or x_t[2] is None):
        raise ValueError("grouped columns and columns of one group")
    E, pstart = 0, None
    if starts is not None:
        E = starts.shape[0] - 1
        pstart = _need(starts, "starts", torch.int32, (E + 1,), dev)
        _need(x_t[2], "x_t.starts", torch.int32, (E + 1,), dev)
    out, pout, f32 = _result(out, dtype, (E, N, K) if starts is not None else (N, K), dev)
    if P == 0:
        return out.zero_()
    ws = _sized(ws, _lib.MOE_SCALED_WS_BYTES, "moe_scaled_weight_gradient", dev)
    _lib.check(_on(dev, _lib.load().moe_scaled_weight_gradient, N, K, P, E, fa, fb, f32, pa, psa, pb, psb, pstart, pout,
                   ws.ptr, ws.nbytes), "moe_scaled_weight_gradient")
    return out
