"""TrainStack refuses parameters that do not fit its layers when it is made (no GPU
is reached)."""
import types

import pytest
import torch

from group_limited_routing_gb300 import moe, train


def layers(*cfgs):
    return [types.SimpleNamespace(cfg=c, device=torch.device("cpu")) for c in cfgs]


CFG = moe.MoeConfig(T=60, H=256)
OK = dict(layers=layers(CFG, CFG), w_pre=(3, 256), w_post=(2, 256), gate=(2, 3, 256))


@pytest.mark.parametrize("bad", [
    dict(layers=[]),
    dict(layers=layers(CFG, moe.MoeConfig(T=60, H=256, rsf=1.0))),      # whose weights' gradient differs
    dict(layers=layers(CFG, moe.MoeConfig(T=60, H=256, k=4))),
    dict(w_pre=(2, 256)), dict(w_pre=(4, 256)), dict(w_pre=(3, 128)), dict(w_post=(3, 256)), dict(w_post=(2, 512)),
    dict(gate=(3, 256)), dict(gate=(2, 128)), dict(gate=(1, 3, 256)), dict(gate=(2, 7, 256)), dict(gate=(2, 0, 256)),
    dict(gate=(2,)),
])
def test_refusals(bad):
    a = {**OK, **bad}
    with pytest.raises(ValueError):
        train.TrainStack(a["layers"], None, torch.ones(a["w_pre"]), torch.ones(a["w_post"]), torch.ones(a["gate"]))


@pytest.mark.parametrize("gate", [(2, 256), (2, 1, 256), (2, 3, 256), (2, 60, 256)])
def test_what_fits_is_taken(monkeypatch, gate):
    monkeypatch.setattr(moe, "SizedWorkspace", lambda nbytes, what, device=None: None)
    step = train.TrainStack(OK["layers"], None, torch.ones(3, 256), torch.ones(2, 256), torch.ones(gate))
    assert step.gate.shape == (2, gate[1] if len(gate) == 3 else 1, 256)
