"""The AdamW step against its formula in fp32 as numpy computes it on the CPU, where
every operation is rounded by itself: over the whole range of fp32, and to the bit."""
import math

import numpy as np
import pytest
import torch

from group_limited_routing_gb300 import optim

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
f = np.float32
MAX = np.finfo(f).max


def on(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def host(t):
    return t.detach().float().cpu().numpy()


def formula(p, g, m, v, t, lr, b1, b2, eps, decay):
    """(p, m, v, root) after step t, each operation rounded to fp32."""
    with np.errstate(all="ignore"):
        m = m * f(b1) + g * f(1 - b1)
        v = v * f(b2) + (g * g) * f(1 - b2)
        root = np.sqrt(v)
        den = root * f(1 / math.sqrt(1 - b2 ** t)) + f(eps)
        p = p * f(1 - lr * decay) - (m / den) * f(lr / (1 - b1 ** t))
    assert p.dtype == m.dtype == root.dtype == f
    return p, m, v, root


def gradient_sizes(n, seed, lo, hi):
    """n values with a power of two between 2^lo and 2^hi for each block of 128."""
    rng = np.random.default_rng(seed)
    size = np.exp2(rng.uniform(lo, hi, -(-n // 128))).repeat(128)[:n]
    return (rng.standard_normal(n) * size).astype(f)


def stepped(p, g, m, v, lr, b1, b2, eps, decay=0.0, step=0):
    """(p, m, v) of a step with states in 32 bits."""
    state = dict(m=[on(m)], v=[on(v)])
    tp = on(p)
    optim.AdamW([tp], lr=lr, betas=(b1, b2), eps=eps, weight_decay=decay, step=step, state=state).step([on(g)])
    return host(tp), host(state["m"][0]), host(state["v"][0])


@pytest.mark.parametrize("lo,hi", [(-16, 0), (-45, 60)])
def test_moments_are_rounded_operation_by_operation(lo, hi):
    n, b1, b2 = 200003, 0.9, 0.999
    p, g = gradient_sizes(n, 4, -6, 0), gradient_sizes(n, 5, lo, hi)
    m, v = gradient_sizes(n, 6, lo, hi), np.square(gradient_sizes(n, 7, max(lo, -40), hi))
    got = stepped(p, g, m, v, 1e-3, b1, b2, 1e-8)
    want = formula(p, g, m, v, 1, 1e-3, b1, b2, 1e-8, 0.0)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[2], want[2])
