"""A wait that runs out in a product of the training operators: the loader
withholds every copy, the first wait gives up after 50 ms, the kernel winds
down by itself, MOE_STATUS_TIMEOUT is reported, and the next call is right."""
import time

import pytest
import torch

from group_limited_routing_gb300 import _lib, moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


def sabotaged(call, launches=1):
    lib = _lib.load()
    assert lib.moe_debug_inject_timeout(launches) == _lib.MOE_OK
    try:
        t0 = time.time()
        call()
        torch.cuda.synchronize()
        assert time.time() - t0 < 10.0
    finally:
        lib.moe_debug_inject_timeout(0)


@pytest.mark.parametrize("T", [20, 300])       # the few-row ring and the full one
def test_loss(T):
    g = torch.Generator().manual_seed(1)
    h = torch.randn(T, 256, generator=g).bfloat16().to(DEV)
    W = (torch.randn(2000, 256, generator=g) * 0.05).bfloat16().to(DEV)
    t = torch.randint(0, 2000, (T,), generator=g).to(DEV)
    d = torch.full((T,), 1.0 / T, device=DEV)
    ws, wb = moe.vocab_loss_workspace(T, 256, 2000), moe.vocab_loss_workspace(T, 256, 2000, backward=True)
    good, lse = moe.vocab_loss(h, W, t, ws=ws)
    grad = moe.vocab_loss_backward(h, W, t, lse, d, ws=wb)
    sabotaged(lambda: moe.vocab_loss(h, W, t, ws=ws))
    assert ws.status() == _lib.MOE_STATUS_TIMEOUT
    assert torch.equal(moe.vocab_loss(h, W, t, ws=ws)[0], good) and ws.status() == 0
    sabotaged(lambda: moe.vocab_loss_backward(h, W, t, lse, d, ws=wb), launches=3)
    assert wb.status() == _lib.MOE_STATUS_TIMEOUT
    again = moe.vocab_loss_backward(h, W, t, lse, d, ws=wb)
    assert wb.status() == 0 and all(torch.equal(again[k], grad[k]) for k in grad)


def test_route_backward():
    g = torch.Generator().manual_seed(2)
    cfg = moe.MoeConfig(T=300, H=512)
    x = torch.randn(300, 512, generator=g).bfloat16().to(DEV)
    W = (torch.randn(256, 512, generator=g) * 0.04).to(DEV)
    idx = moe.route(cfg, x, W)[0]
    d_w = torch.randn(300, 8, generator=g).to(DEV)
    ws = moe.route_backward_workspace(cfg)
    call = lambda: moe.route_backward(cfg, x, W, idx, d_w, d_hidden_add=x, ws=ws)  # noqa: E731
    good = call()
    sabotaged(call, launches=2)
    assert ws.status() == _lib.MOE_STATUS_TIMEOUT
    again = call()
    assert ws.status() == 0 and all(torch.equal(again[k], good[k]) for k in good)
