"""The gradients' norm over the whole range of fp32, against sums in 64 bits."""
import math

import pytest
import torch

from group_limited_routing_gb300 import optim

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.bfloat16, torch.float32]


def grads(size, dtype, sizes, seed=1):
    """A part of the values at `size`, the others zero."""
    g = torch.Generator(DEV).manual_seed(seed)
    out = []
    for n in sizes:
        x = torch.randn(n, device=DEV, generator=g, dtype=torch.float64) * size
        x[torch.rand(n, device=DEV, generator=g) < 0.5] = 0
        out.append(x.to(dtype))
    return out


def check(tensors, max_norm=1.0):
    want = math.sqrt(math.fsum(float(t.double().square().sum()) for t in tensors))
    norm, scale = optim.grad_norm(tensors, max_norm=max_norm)
    # fp32 sums of up to 32 squares, the rest in 64 bits; the norm rounded once.  A norm
    # under 2^-126 is rounded to a multiple of 2^-149.
    assert abs(norm.item() - want) <= want * 2.0 ** -22 + 2.0 ** -150, (norm.item(), want)
    limit = min(1.0, max_norm / want) if want else 1.0
    assert abs(scale.item() - limit) <= limit * 2.0 ** -22
    return want


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("exponent", [120, 80, 64, 60, 0, -40, -45, -50, -60, -63, -66, -70, -76, -100, -120, -126])
def test_norm_of_every_size(exponent, dtype):
    check(grads(2.0 ** exponent, dtype, [8192, 3 * 8192, 8193, 100, 1]))


@pytest.mark.parametrize("dtype", TYPES)
def test_sizes_side_by_side(dtype):
    tiny, huge, plain = grads(2.0 ** -80, dtype, [8192, 50], 2), grads(2.0 ** 70, dtype, [8192, 50], 3), \
        grads(1.0, dtype, [8192, 50], 4)
    zero = [torch.zeros(n, dtype=dtype, device=DEV) for n in (8192, 50)]
    for tensors in (tiny + zero, tiny + plain, tiny + huge, zero + huge + plain, zero):
        check(tensors)
    one = torch.zeros(8192, dtype=dtype, device=DEV)
    one[1::8] = 2.0 ** -72                       # a lane's squares vanish but for one's
    one[2] = 2.0 ** -40
    check([one])
    # views that start anywhere
    check([t[1:] for t in tiny + huge])


def test_a_gradient_of_a_large_norm_is_scaled_and_stepped():
    g = [torch.full((300,), 1e20, device=DEV)]
    want = check(g)
    p = torch.zeros(300, device=DEV)
    norm, scale = optim.grad_norm(g)
    optim.AdamW([p], lr=0.1, weight_decay=0.0).step(g, grad_scale=scale)
    first = 1e20 / want                          # the first step: lr g / (|g| + eps)
    assert bool((p.double() + 0.1 * first / (first + 1e-8)).abs().max() <= 0.1 * 2.0 ** -20)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("at", [(0, 100), (1, 7)])
def test_infinities_and_nan(at, bad, dtype):
    g = grads(1.0, dtype, [8192, 50])
    g[at[0]][at[1]] = bad
    norm, scale = optim.grad_norm(g)
    assert math.isnan(scale.item())
    assert math.isnan(norm.item()) if math.isnan(bad) else norm.item() == math.inf


def test_a_norm_past_the_largest_number():
    """3e38 sixteen times: the norm is 1.2e39."""
    norm, scale = optim.grad_norm([torch.full((16,), 3e38, device=DEV)])
    assert norm.item() == math.inf and math.isnan(scale.item())
    check([torch.full((1,), 3e38, device=DEV)])
