"""MoeConfig.c(): the caller's own structure each time."""
import copy
import pickle

from group_limited_routing_gb300 import moe


def test_a_changed_structure_leaves_the_configuration_alone():
    cfg = moe.MoeConfig(T=5, rsf=1.5)
    c = cfg.c()
    c.T, c.rsf = 9, 0.0
    assert (cfg.c().T, cfg.c().rsf) == (5, 1.5)
    assert cfg.ref()._obj.T == 5


def test_copies_and_equality():
    cfg = moe.MoeConfig(T=5)
    cfg.ref()
    for other in (copy.copy(cfg), copy.deepcopy(cfg), pickle.loads(pickle.dumps(cfg)), cfg.with_T(5)):
        assert other == cfg and hash(other) == hash(cfg) and other.ref()._obj.T == 5
    assert cfg.with_T(7).ref()._obj.T == 7 and cfg.ref()._obj.T == 5
