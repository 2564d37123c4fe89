"""optim.AdamW refuses what no step could take when it is made (on the CPU: no kernel
runs)."""
import math
import types

import pytest
import torch

from group_limited_routing_gb300 import build, optim, train


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def params(*sizes):
    return [torch.zeros(n) for n in sizes or (8, 3)]


@pytest.mark.parametrize("kw", [
    dict(lr=math.nan), dict(lr=math.inf), dict(betas=(1.0, 0.999)), dict(betas=(0.9, 1.0)), dict(betas=(-0.1, 0.9)),
    dict(betas=(0.9, math.nan)), dict(betas=(0.9,)), dict(eps=-1e-8), dict(eps=math.nan), dict(eps=math.inf),
    dict(weight_decay=-0.1), dict(weight_decay=[0.1, math.nan]), dict(weight_decay=math.inf), dict(step=-1)])
def test_numbers_that_no_step_takes(kw):
    with pytest.raises(ValueError, match=next(iter(kw))):
        optim.AdamW(params(), **kw)


@pytest.mark.parametrize("kw", [dict(lr=0.0), dict(lr=-1e-3), dict(betas=[0.0, 0.0]), dict(eps=0), dict(weight_decay=[0, 0.1]),
                                dict(step=7)])
def test_numbers_at_the_border(kw):
    opt = optim.AdamW(params(), **kw)
    assert opt.step_number == kw.get("step", 0)


def test_tensors_that_share_memory():
    whole = torch.zeros(100)
    for bad in ([whole, torch.zeros(3), whole], [whole[:60], whole[59:]], [whole, whole[10:20]]):
        with pytest.raises(ValueError, match=r"params\[\d\] and params\[\d\] overlap"):
            optim.AdamW(bad)
    optim.AdamW([whole[:60], whole[60:], whole[60:60]])
    m = [torch.zeros(8), torch.zeros(3)]
    with pytest.raises(ValueError, match="overlap"):
        optim.AdamW(params(), state=dict(m=m, v=[m[0], torch.zeros(3)]))
    p = params()
    with pytest.raises(ValueError, match="overlap"):
        optim.AdamW(p, state=dict(m=m, v=[torch.zeros(8), p[1]]))
    p = [torch.zeros(8, dtype=torch.bfloat16), torch.zeros(3)]
    with pytest.raises(ValueError, match="overlap"):
        optim.AdamW(p, master=True, state=dict(m=m, v=[torch.zeros(8), torch.zeros(3)], master=[m[0], None]))


def test_layers_that_share_a_weight():
    names = [name for name, _ in train.TrainStack._LAYER]
    stack = train.TrainStack.__new__(train.TrainStack)
    stack.layers = [types.SimpleNamespace(**{name: torch.zeros(4) for name in names}) for _ in range(3)]
    stack.head = types.SimpleNamespace(W_vocab=torch.zeros(4))
    stack.w_pre = stack.w_post = stack.gate = None
    assert len(stack.parameters()) == 4 + 3 * len(names)
    stack.layers[2].W_down = stack.layers[0].W_down
    with pytest.raises(ValueError, match="W_down of layer 2"):
        stack.parameters()
    with pytest.raises(ValueError, match="W_down of layer 2"):
        stack.gradients({})
