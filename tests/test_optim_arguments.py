"""optim.AdamW refuses what no step could take when it is made (on the CPU: no kernel
runs)."""
import math

import pytest
import torch

from group_limited_routing_gb300 import build, optim


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
