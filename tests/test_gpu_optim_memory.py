"""AdamW whose parameters or states are given other memory between steps, and steps
that are refused: what is refused changes nothing, what is followed gives the same
results."""
import math

import pytest
import torch

from group_limited_routing_gb300 import optim

pytestmark = pytest.mark.gpu
DEV = "cuda"
SIZES = [300, 8, 129]


def tensors(seed, dtype=torch.float32):
    g = torch.Generator(DEV).manual_seed(seed)
    return [torch.randn(n, device=DEV, generator=g).to(dtype) for n in SIZES]


def test_a_failed_change_of_memory_leaves_no_parameter_behind():
    a, b, grads = tensors(1), tensors(1), tensors(2)
    oa, ob = optim.AdamW(a, lr=0.1), optim.AdamW(b, lr=0.1)
    old = b[1].data
    b[1].data = torch.zeros(9, device=DEV)
    with pytest.raises(ValueError, match="params"):
        ob.step(grads)
    b[1].data = old
    for t in range(2):
        oa.step(grads)
        ob.step(grads)
        for x, y in zip(a, b):
            assert torch.equal(x, y)
        for p in b:
            p.data = p.data.clone()
