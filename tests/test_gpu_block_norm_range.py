"""Gradient of block_norm where 1 / RMS is large: rows of zeros with a tiny eps,
and tiny rows with none.  sigma = 1 / sqrt(mean r^2 + eps) is 1e14 to 1e15 there:
sigma^2 fits fp32, sigma^3 does not, and the formula holds no sigma^3.

Tolerances: test_gpu_block_norm's, element by element (fp32 arithmetic whose
relative errors do not depend on the scale)."""
import pytest
import torch

from group_limited_routing_gb300 import moe
from test_gpu_block_norm import check, inputs

pytestmark = pytest.mark.gpu


def gradients(d, eps, has_y=True):
    g = moe.block_norm_backward(d["x"], d["y"], d["gate"], d["w_post"], d["w_pre"], d["d_r"], d["d_n"], alpha=0.9,
                                eps=eps)
    assert all(t.isfinite().all() for t in g.values())
    check(g, d, 0.9, eps, has_y)


@pytest.mark.parametrize("H", [256, 2048, 6000])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [True, False])
def test_rows_of_zeros_with_a_tiny_eps(H, stream, block):
    d = inputs(40, H, 4 if block else None, stream, seed=H)
    for name in ("x", "y"):
        d[name][5] = 0
        d[name][39] = 0
    if not block:
        d.update(y=None, w_post=None)
    gradients(d, 1e-30, block)


@pytest.mark.parametrize("H", [256, 2048, 6000])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_tiny_rows_without_eps(H, stream):
    d = inputs(33, H, None, stream, seed=H + 1)
    d.update(y=None, w_post=None)
    d["x"][::3] *= 1e-14
    gradients(d, 0.0, has_y=False)


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_tiny_stream_and_gate_without_eps(stream):
    d = inputs(36, 512, 4, stream, seed=17)
    d["x"] *= 1e-14
    d["gate"] *= 1e-14
    gradients(d, 0.0)
