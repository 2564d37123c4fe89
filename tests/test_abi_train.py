"""The training operators' entry points refuse wrong arguments on the host,
before any CUDA call (so these run without a GPU)."""
import ctypes

import pytest

from group_limited_routing_gb300 import _lib, build

A = 1 << 20          # a fake aligned address: never dereferenced, the checks fail first
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


# ------------------------------------------------------------- block norm
def norm(lib, T=64, H=2048, groups=1, f32=0, x=A, y=A, gate=A, post=A, pre=A, alpha=1.0, eps=1e-6, r=A, n=A):
    return lib.moe_block_norm(T, H, groups, f32, x, y, gate, post, pre, alpha, eps, r, n, None)


def norm_bwd(lib, T=64, H=2048, groups=1, f32=0, x=A, y=A, gate=A, post=A, pre=A, alpha=1.0, eps=1e-6, d_r=A, d_n=A,
             d_x=A, d_y=A, d_gate=A, d_post=A, d_pre=A, ws=A, ws_bytes=BIG):
    return lib.moe_block_norm_backward(T, H, groups, f32, x, y, gate, post, pre, alpha, eps, d_r, d_n, d_x, d_y,
                                       d_gate, d_post, d_pre, ws, ws_bytes, None)


SHAPES = [
    (dict(T=0), _lib.MOE_ERR_INVALID_ARG), (dict(H=0), _lib.MOE_ERR_INVALID_ARG),
    (dict(groups=0), _lib.MOE_ERR_INVALID_ARG), (dict(T=64, groups=3), _lib.MOE_ERR_INVALID_ARG),
    (dict(f32=2), _lib.MOE_ERR_INVALID_ARG), (dict(eps=-1e-6), _lib.MOE_ERR_INVALID_ARG),
    (dict(eps=float("nan")), _lib.MOE_ERR_INVALID_ARG), (dict(alpha=float("inf")), _lib.MOE_ERR_INVALID_ARG),
    (dict(H=2044), _lib.MOE_ERR_UNSUPPORTED_SHAPE), (dict(H=8200), _lib.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(T=(1 << 24) + 1), _lib.MOE_ERR_UNSUPPORTED_SHAPE), (dict(x=None), _lib.MOE_ERR_INVALID_ARG),
    (dict(x=A + 8), _lib.MOE_ERR_MISALIGNED), (dict(gate=A + 4), _lib.MOE_ERR_MISALIGNED),
]


@pytest.mark.parametrize("kw,code", SHAPES + [
    (dict(n=None), _lib.MOE_ERR_INVALID_ARG), (dict(r=None), _lib.MOE_ERR_INVALID_ARG),
    (dict(y=None), _lib.MOE_ERR_INVALID_ARG),                       # a gate without a block output
    (dict(n=A + 2), _lib.MOE_ERR_MISALIGNED),
])
def test_block_norm_refusals(lib, kw, code):
    assert norm(lib, **kw) == code


@pytest.mark.parametrize("kw,code", SHAPES + [
    (dict(d_n=None), _lib.MOE_ERR_INVALID_ARG), (dict(d_x=None), _lib.MOE_ERR_INVALID_ARG),
    (dict(d_y=None), _lib.MOE_ERR_INVALID_ARG), (dict(ws=None), _lib.MOE_ERR_INVALID_ARG),
    (dict(y=None, gate=None, post=None), _lib.MOE_ERR_INVALID_ARG),  # a gradient of an absent block output
    (dict(ws_bytes=1024), _lib.MOE_ERR_WORKSPACE_TOO_SMALL), (dict(ws=A + 16), _lib.MOE_ERR_MISALIGNED),
    (dict(d_r=A + 2), _lib.MOE_ERR_MISALIGNED),
])
def test_block_norm_backward_refusals(lib, kw, code):
    assert norm_bwd(lib, **kw) == code


def test_block_norm_workspace(lib):
    n = lib.moe_block_norm_workspace_bytes(64, 2048, 1)
    assert n % 256 == 0 and n >= 256 + 2 * 64 * 2048 * 4         # a partial sum per row-block of each column
    assert lib.moe_block_norm_workspace_bytes(64, 2048, 64) >= n  # a gate per token
    assert lib.moe_block_norm_workspace_bytes(64, 2048, 3) == 0
    assert lib.moe_block_norm_workspace_bytes(64, 2044, 1) == 0


# ------------------------------------------------------- vocabulary loss
def loss(lib, T=64, H=2048, V=1000, hidden=A, W=A, target=A, bits=64, ignore=-100, out=A, lse=A, ws=A, ws_bytes=BIG):
    return lib.moe_vocab_loss(T, H, V, hidden, W, target, bits, ignore, out, lse, ws, ws_bytes, None)


def loss_bwd(lib, T=64, H=2048, V=1000, hidden=A, W=A, target=A, bits=64, ignore=-100, lse=A, d_loss=A, d_hidden=A,
             dW=A, ws=A, ws_bytes=BIG):
    return lib.moe_vocab_loss_backward(T, H, V, hidden, W, target, bits, ignore, lse, d_loss, d_hidden, dW, ws,
                                       ws_bytes, None)


VOCAB = [
    (dict(T=-1), _lib.MOE_ERR_INVALID_ARG), (dict(H=0), _lib.MOE_ERR_INVALID_ARG), (dict(V=0), _lib.MOE_ERR_INVALID_ARG),
    (dict(bits=16), _lib.MOE_ERR_INVALID_ARG), (dict(H=2044), _lib.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(H=(1 << 16) + 8), _lib.MOE_ERR_UNSUPPORTED_SHAPE), (dict(T=(1 << 24) + 1), _lib.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(V=(1 << 24) + 1), _lib.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(T=1 << 24, V=1 << 24), _lib.MOE_ERR_UNSUPPORTED_SHAPE), (dict(hidden=None), _lib.MOE_ERR_INVALID_ARG),
    (dict(W=None), _lib.MOE_ERR_INVALID_ARG), (dict(target=None), _lib.MOE_ERR_INVALID_ARG),
    (dict(ws=None), _lib.MOE_ERR_INVALID_ARG), (dict(ws_bytes=4096), _lib.MOE_ERR_WORKSPACE_TOO_SMALL),
    (dict(ws=A + 128), _lib.MOE_ERR_MISALIGNED), (dict(hidden=A + 8), _lib.MOE_ERR_MISALIGNED),
    (dict(W=A + 2), _lib.MOE_ERR_MISALIGNED), (dict(target=A + 4), _lib.MOE_ERR_MISALIGNED),
    (dict(lse=None), _lib.MOE_ERR_INVALID_ARG), (dict(lse=A + 1), _lib.MOE_ERR_MISALIGNED),
]


@pytest.mark.parametrize("kw,code", VOCAB + [(dict(out=None), _lib.MOE_ERR_INVALID_ARG)])
def test_vocab_loss_refusals(lib, kw, code):
    assert loss(lib, **kw) == code


@pytest.mark.parametrize("kw,code", VOCAB + [
    (dict(d_loss=None), _lib.MOE_ERR_INVALID_ARG), (dict(d_hidden=None), _lib.MOE_ERR_INVALID_ARG),
    (dict(dW=None), _lib.MOE_ERR_INVALID_ARG), (dict(dW=A + 8), _lib.MOE_ERR_MISALIGNED),
])
def test_vocab_loss_backward_refusals(lib, kw, code):
    assert loss_bwd(lib, **kw) == code


def test_vocab_loss_of_no_rows_touches_nothing(lib):
    assert loss(lib, T=0, hidden=None, target=None, out=None, lse=None, ws=None) == _lib.MOE_OK


def test_vocab_loss_workspace(lib):
    size = lib.moe_vocab_loss_workspace_bytes
    # forward: a pair of floats per row and 256 columns, never the logits
    assert 0 < size(8192, 2048, 131072, 0) < 8192 * 131072 // 8
    # backward: dlogits of a piece of the vocabulary, at most 1 GiB beside the rows' buffers
    rows = 8192 * 2048 * 2 + 16 * 8192 * 2048 * 4
    assert 0 < size(8192, 2048, 131072, 1) < (1 << 30) + rows + (1 << 20)
    assert size(8192, 2044, 131072, 0) == 0 and size(8192, 2048, 0, 1) == 0
    assert size(0, 64, 100, 1) > 0


# --------------------------------------------------- the router's gradient
def cfg(**kw):
    base = dict(T=64, H=2048, E=256, n_group=8, topk_group=4, k=8, I=512, Is=512, rsf=2.5, eps=1e-20)
    base.update(kw)
    return _lib.MoeCfg(*[base[n] for n in ("T", "H", "E", "n_group", "topk_group", "k", "I", "Is")],
                       base["rsf"], base["eps"])


def route_bwd(lib, c, hidden=A, W=A, split=None, idx=A, d_w=A, counts=A, d_aux=A, add=A, d_hidden=A, dW=A, ws=A,
              ws_bytes=BIG):
    return lib.moe_route_backward(ctypes.byref(c), hidden, W, split, idx, d_w, counts, d_aux, add, d_hidden, dW, ws,
                                  ws_bytes, None)


@pytest.mark.parametrize("c,kw,code", [
    (dict(T=0), {}, _lib.MOE_ERR_INVALID_ARG), (dict(H=2000), {}, _lib.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(k=129), {}, _lib.MOE_ERR_INVALID_ARG), (dict(E=512, n_group=16), {}, _lib.MOE_ERR_UNSUPPORTED_SHAPE),
    ({}, dict(hidden=None), _lib.MOE_ERR_INVALID_ARG), ({}, dict(idx=None), _lib.MOE_ERR_INVALID_ARG),
    ({}, dict(d_w=None), _lib.MOE_ERR_INVALID_ARG), ({}, dict(counts=None), _lib.MOE_ERR_INVALID_ARG),
    ({}, dict(d_hidden=None), _lib.MOE_ERR_INVALID_ARG), ({}, dict(dW=None), _lib.MOE_ERR_INVALID_ARG),
    ({}, dict(ws=None), _lib.MOE_ERR_INVALID_ARG), ({}, dict(ws_bytes=1 << 16), _lib.MOE_ERR_WORKSPACE_TOO_SMALL),
    ({}, dict(ws=A + 16), _lib.MOE_ERR_MISALIGNED), ({}, dict(hidden=A + 8), _lib.MOE_ERR_MISALIGNED),
    ({}, dict(split=A + 8), _lib.MOE_ERR_MISALIGNED), ({}, dict(add=A + 2), _lib.MOE_ERR_MISALIGNED),
    ({}, dict(dW=A + 8), _lib.MOE_ERR_MISALIGNED), ({}, dict(idx=A + 2), _lib.MOE_ERR_MISALIGNED),
])
def test_route_backward_refusals(lib, c, kw, code):
    assert route_bwd(lib, cfg(**c), **kw) == code


def test_route_backward_workspace(lib):
    size = lib.moe_route_backward_workspace_bytes
    assert size(ctypes.byref(cfg())) % 256 == 0
    assert size(ctypes.byref(cfg())) > 3 * 256 * 2048 * 2 + 3 * 64 * 256 * 2 + 256 * 2048 * 4
    assert size(ctypes.byref(cfg(H=2000))) == 0 and size(None) == 0
