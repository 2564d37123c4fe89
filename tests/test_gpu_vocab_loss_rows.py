"""vocab_loss where a row's result might follow its company."""
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
