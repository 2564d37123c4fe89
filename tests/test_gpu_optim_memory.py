"""AdamW whose parameters or states are given other memory between steps, and steps
that are refused: what is refused changes nothing, what is followed gives the same
results."""
import math

import pytest
import torch

from group_limited_routing_gb300 import _lib, optim

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


@pytest.mark.parametrize("bits,dtype,master", [(32, torch.float32, False), (32, torch.bfloat16, True), (8, torch.float32, False),
                                               (8, torch.bfloat16, True)])
def test_states_given_other_memory(bits, dtype, master):
    """Loaded states take the old ones' places, which nobody writes any more; so do
    states whose memory was exchanged below them."""
    a, b, grads = tensors(1, dtype), tensors(1, dtype), tensors(2)
    kw = dict(lr=0.1, state_bits=bits, master=master, seed=3)
    oa, ob = optim.AdamW(a, **kw), optim.AdamW(b, **kw)
    raw = lambda t: t.view(torch.uint8)  # noqa: E731
    for way in range(3):
        if way:
            old = [t for held in ob.state.values() for t in held]
            if way == 1:                         # each list's tensors replaced, one by one
                for held in ob.state.values():
                    for i in range(len(SIZES)):
                        held[i] = held[i].clone()
            else:                                # (a tensor keeps its identity)
                for t in old:
                    t.data = t.data.clone()
                old = []
            kept = [raw(t).clone() for t in old]
        oa.step(grads)
        ob.step(grads)
        for x, y in zip(a, b):
            assert torch.equal(x, y)
        for name in oa.state:
            for x, y in zip(oa.state[name], ob.state[name]):
                assert torch.equal(raw(x), raw(y))
        if way:
            for t, k in zip(old, kept):
                assert torch.equal(raw(t), k)
    ob.state = {name: [t.clone() for t in held] for name, held in ob.state.items()}    # a whole new dict
    oa.step(grads)
    ob.step(grads)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_states_that_do_not_fit_are_refused():
    p, grads = tensors(1), tensors(2)
    opt = optim.AdamW(p, lr=0.1)
    before, m = [x.clone() for x in p], opt.state["m"][1]
    for bad, error in ((torch.zeros(9, device=DEV), ValueError), (torch.zeros(8, device=DEV, dtype=torch.float64), TypeError),
                       (torch.zeros(8), ValueError), (None, TypeError)):
        opt.state["m"][1] = bad
        with pytest.raises(error, match="state"):
            opt.step(grads)
    opt.state["m"][1] = m
    opt.state["v"].append(m)
    with pytest.raises(ValueError, match="state"):
        opt.step(grads)
    opt.state["v"].pop()
    assert opt.step_number == 0 and all(torch.equal(x, y) for x, y in zip(before, p))
    opt.step(grads)
    assert opt.step_number == 1 and not any(torch.equal(x, y) for x, y in zip(before, p))


@pytest.mark.parametrize("capturable", [False, True])
def test_a_step_that_the_library_refuses_does_not_count(capturable, monkeypatch):
    a, b, grads = tensors(1), tensors(1), tensors(2)
    oa, ob = [optim.AdamW(p, lr=0.1, capturable=capturable) for p in (a, b)]
    with monkeypatch.context() as m:
        m.setattr(_lib.load(), "moe_adamw", lambda *_: _lib.MOE_ERR_INVALID_ARG)
        for kw in ({}, dict(lr=0.5)):
            with pytest.raises(_lib.MoeError):
                ob.step(grads, **kw)
    ob.lr = math.nan
    with pytest.raises(ValueError, match="lr"):
        ob.step(grads)
    ob.lr = 0.1
    assert ob.step_number == 0
    if capturable:
        assert ob.step_count.item() == 0 and ob.lr_now.item() == oa.lr_now.item()
    for opt in (oa, ob):
        opt.step(grads)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
