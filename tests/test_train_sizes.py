"""Sizes of the training step's workspaces (no GPU: the allocation is replaced)."""
import types

import pytest
import torch

from group_limited_routing_gb300 import _lib, build, moe, train


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


@pytest.fixture
def stack(lib, monkeypatch):
    """A TrainStack of one layer whose workspaces are sizes only."""
    monkeypatch.setattr(moe, "SizedWorkspace",
                        lambda nbytes, what, device=None: types.SimpleNamespace(nbytes=int(nbytes)))

    def make(T, H, groups):
        layer = types.SimpleNamespace(cfg=moe.MoeConfig(T=T, H=H), device=torch.device("cpu"))
        return train.TrainStack([layer], None, torch.ones(2, H), torch.ones(1, H), torch.ones(1, groups, H))

    return make


@pytest.mark.parametrize("H", [256, 512, 1536, 2048, 4096])
@pytest.mark.parametrize("groups", [1, 2, 3, 5, 6, 7, 12, 64])
def test_norm_workspace_covers_the_gated_norms_and_the_first(lib, stack, H, groups):
    """The norms behind the layers have a gate row per group, the one in front of the
    first none: its plan is that of one group, whose partial sums may be more."""
    for T in (groups, 60 * groups, 840 * groups, 1365 * groups, 4096 * groups):
        nbytes = stack(T, H, groups).ws_norm.nbytes
        for g in (groups, 1):
            need = lib.moe_block_norm_workspace_bytes(T, H, g)
            assert 0 < need <= nbytes, (T, H, g)
