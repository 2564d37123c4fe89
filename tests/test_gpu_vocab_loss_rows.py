"""vocab_loss where a row's result might follow its company: few rows that count
among many that do not, blocks of the vocabulary whose logits are infinite."""
import pytest
import torch

from group_limited_routing_gb300 import moe
from test_gpu_vocab_loss import DEV, IGN, U, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,keep", [(20, 3), (300, 1), (1000, 3), (1000, 8), (3000, 5)])
@pytest.mark.parametrize("H", [2048, 3144])
def test_few_rows_that_count_are_summed_as_few_rows(T, keep, H):
    """Up to 8 rows that count have the accuracy of a call of up to 8 rows, however
    many ignored ones stand beside them.  Against 64 bits: a logit's K is cut into
    parts of 256, each 16 steps of the tensor core off by at most one unit (2 U) of
    the part's magnitudes, then added (half a unit per part); the softmax as in
    test_gpu_vocab_loss.  And the parts being the same, so are the bits."""
    d = inputs(T, H, 3000, seed=T + H + keep)
    on = torch.randperm(T, generator=torch.Generator().manual_seed(keep))[:keep].sort().values.to(DEV)
    target = torch.full_like(d["target"], IGN)
    target[on] = d["target"][on]
    loss, lse = moe.vocab_loss(d["hidden"], d["W"], target)
    alone, alone_lse = moe.vocab_loss(d["hidden"][on].contiguous(), d["W"], d["target"][on].contiguous())
    assert torch.equal(loss[on], alone) and torch.equal(lse[on], alone_lse)
    h, W, t = d["hidden"][on].double(), d["W"].double(), d["target"][on][:, None]
    z = h @ W.t()
    zb = (16 * 2 + H / 256 + 4) * U * (h.abs() @ W.abs().t())
    ref, at = torch.logsumexp(z, 1), z.gather(1, t)[:, 0]
    bound = zb.amax(1) + zb.gather(1, t)[:, 0] + U * (128 + 4 * z.abs().amax(1) + 6 * ref.abs() + at.abs())
    over = ((loss[on].double() - (ref - at)).abs() / bound).max().item()
    assert over <= 1, "loss off by %.3g of its bound" % over



def extreme(T, V, H, level, blocks, value, seed):
    """Logits near `level` (component 1), except in the 128-column blocks listed,
    where component 0 makes them `value` times 1e40: infinite in fp32."""
    g = torch.Generator().manual_seed(seed)
    W = torch.zeros(V, H)
    W[:, 1] = level + torch.randn(V, generator=g)
    h = torch.zeros(T, H)
    h[:, 0] = 1e20
    h[:, 1] = 1.0
    for b in blocks:
        W[128 * b:128 * (b + 1), 0] = value * 1e20
    free = [v for v in range(V) if v // 128 not in blocks]
    target = torch.tensor([free[(7 * t) % len(free)] for t in range(T)])
    return h.bfloat16().to(DEV), W.bfloat16().to(DEV), target.to(DEV), torch.tensor(free, device=DEV)


@pytest.mark.parametrize("T", [3, 20, 200])
@pytest.mark.parametrize("level", [-300.0, -100.0, 5.0, 200.0])
@pytest.mark.parametrize("blocks", [[0], [3], [1, 2], [0, 4]])
def test_blocks_of_minus_infinity_take_nothing(T, level, blocks):
    """Logits of minus infinity are no part of the sum, whatever the others' level:
    (128 + 4 |z| + 4 |lse|) half-steps, as for any row, the logits being exact."""
    h, W, target, free = extreme(T, 600, 64, level, blocks, -1.0, seed=T)
    loss, lse = moe.vocab_loss(h, W, target)
    z = h[:, 1:].double() @ W[free, 1:].double().t()
    ref, at = torch.logsumexp(z, 1), (h[:, 1:].double() * W[target, 1:].double()).sum(1)
    bound = U * (128 + 4 * z.abs().amax(1) + 4 * ref.abs())
    assert ((lse.double() - ref).abs() <= bound).all()
    assert ((loss.double() - (ref - at)).abs() <= bound + U * (at.abs() + ref.abs())).all()
    # their probability is 0 in the gradient: every element of it is finite
    d = torch.full((T,), 1.0 / T, device=DEV)
    g = moe.vocab_loss_backward(h, W, target, lse, d)
    assert all(t.isfinite().all() for t in g.values())
    inside = [128 * b for b in blocks]
    assert not g["dW_vocab"][inside].any()


@pytest.mark.parametrize("T", [3, 20, 200])
@pytest.mark.parametrize("level", [-300.0, 5.0, 300.0])
@pytest.mark.parametrize("blocks", [[0], [3], [0, 4]])
def test_blocks_of_plus_infinity_give_infinity(T, level, blocks):
    """lse is infinite and so is the loss of a finite target, as the formula has
    it (not NaN), whatever the other logits' level."""
    h, W, target, _ = extreme(T, 600, 64, level, blocks, 1.0, seed=T)
    loss, lse = moe.vocab_loss(h, W, target)
    assert (lse == float("inf")).all() and (loss == float("inf")).all()


def test_rows_of_nothing_but_minus_infinity():
    """log of an empty sum, as logsumexp has it; NaN beside minus infinity stays."""
    h = torch.full((5, 64), 0.0)
    h[:, 0] = 1e20
    W = torch.zeros(256, 64)
    W[:, 0] = -1e20
    h, W, target = h.bfloat16().to(DEV), W.bfloat16().to(DEV), torch.arange(5, device=DEV)
    loss, lse = moe.vocab_loss(h, W, target)
    assert (lse == float("-inf")).all() and torch.isnan(loss).all()
    W[200, 3] = float("nan")
    loss, lse = moe.vocab_loss(h, W, target)
    assert torch.isnan(lse).all()
