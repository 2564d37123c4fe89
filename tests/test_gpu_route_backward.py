"""route_backward on the GPU against the formula in 64 bits (autograd of the
weights and of the balance loss) and against differences.

Tolerances: the logits are within dL = 2e-6 + 2e-6 max|L| of the exact ones (the
router's own bound), a score moves by less than dL of its own size, so a
logit's gradient, a short chain of products and sums of those scores, by less
than (8 dL + 64 half-steps of 2^-24) of the magnitudes it is formed from;
d_hidden adds the products' 2^-16 (parts left out) and its rounding to bf16,
2^-8; dW_router adds the fp32 sums, 3 x 64 steps of 2^-23 within a split of the
tokens and one of 2^-24 per split."""
import pytest
import torch

from group_limited_routing_gb300 import _lib, moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def inputs(T, H, E=256, k=8, seed=0, keep=None):
    g = torch.Generator().manual_seed(seed)
    cfg = moe.MoeConfig(T=T, H=H, E=E, n_group=E // 32, topk_group=keep or max(1, E // 64), k=k)
    d = dict(hidden=torch.randn(T, H, generator=g).bfloat16().to(DEV),
             W=(torch.randn(E, H, generator=g) * (1.0 / H ** 0.5)).to(DEV),
             d_w=torch.randn(T, k, generator=g).to(DEV), d_aux=torch.tensor([0.7], device=DEV),
             add=torch.randn(T, H, generator=g).bfloat16().to(DEV))
    d["idx"], _, d["counts"], _, _ = moe.route(cfg, d["hidden"], d["W"])
    return cfg, d


def reference(cfg, d, aux, idx_ok=None):
    x, W = d["hidden"].double().requires_grad_(), d["W"].double().requires_grad_()
    L = x @ W.t()
    s = torch.sigmoid(L)
    idx = d["idx"].long()
    ok = torch.ones_like(idx, dtype=torch.bool) if idx_ok is None else idx_ok
    idx = torch.where(ok, idx, 0)
    c = torch.where(ok, s.gather(1, idx), 0.0)
    D = c.sum(1, keepdim=True) + cfg.eps
    dw = torch.where(ok, d["d_w"].double(), 0.0)
    total = (c / D * cfg.rsf * dw).sum()
    Z = s.sum(1, keepdim=True)
    f = d["counts"].double() / (cfg.k * cfg.T)
    if aux:
        total = total + d["d_aux"].double()[0] * cfg.E * (f * (s / Z).mean(0)).sum()
    dx, dW = torch.autograd.grad(total, [x, W])
    # magnitudes of dL
    s, c, D, Z = s.detach(), c.detach(), D.detach(), Z.detach()
    m = torch.zeros_like(s).scatter_add_(1, idx, cfg.rsf / D * (dw.abs() + (dw.abs() * c).sum(1, keepdim=True) / D) * ok)
    if aux:
        m = m + d["d_aux"].double()[0] * cfg.E / cfg.T * (f + (f * s).sum(1, keepdim=True) / Z) / Z
    m = m * s * (1 - s)
    rel = 8 * (2e-6 + 2e-6 * L.detach().abs().amax(1, keepdim=True)) + 64 * U
    x, W = x.detach(), W.detach()
    bx = (rel * m) @ W.abs() + 2.0 ** -16 * (m @ W.abs())
    bW = (rel * m).t() @ x.abs() + (3 * 64 * 2 + cfg.T / 1024 + 152) * U * (m.t() @ x.abs())
    return dx, dW, bx, bW


def check(cfg, d, got, aux, add, **kw):
    dx, dW, bx, bW = reference(cfg, d, aux, **kw)
    if add:
        dx = dx + d["add"].double()
    bx = bx + 2.0 ** -8 * dx.abs() + 2 * U * d["add"].double().abs() + 1e-37
    over = ((got["d_hidden"].double() - dx).abs() / bx).max().item()
    assert over <= 1, "d_hidden off by %.3g of its bound" % over
    over = ((got["dW_router"].double() - dW).abs() / (bW + 1e-37)).max().item()
    assert over <= 1, "dW_router off by %.3g of its bound" % over


def run(cfg, d, aux, add, **kw):
    ws = moe.route_backward_workspace(cfg)
    got = moe.route_backward(cfg, d["hidden"], d["W"], d["idx"], d["d_w"], d_aux_loss=d["d_aux"] if aux else None,
                             expert_counts=d["counts"] if aux else None, d_hidden_add=d["add"] if add else None, ws=ws,
                             **kw)
    return got, ws


@pytest.mark.parametrize("T,H,E,k", [
    (1, 64, 256, 8), (2, 2048, 256, 8), (16, 2048, 256, 8), (32, 512, 256, 4), (33, 512, 256, 8), (63, 192, 128, 1),
    (65, 320, 256, 8), (128, 512, 256, 8), (257, 2048, 256, 6), (1000, 1536, 128, 8), (1030, 576, 256, 8),
    (4096, 2048, 256, 8), (20000, 256, 256, 8),
])
@pytest.mark.parametrize("aux,add", [(False, False), (True, True)])
def test_formula(T, H, E, k, aux, add):
    cfg, d = inputs(T, H, E, k, seed=T + H)
    got, ws = run(cfg, d, aux, add)
    assert ws.status() == 0
    check(cfg, d, got, aux, add)


@pytest.mark.parametrize("T,H,E,k", [(34, 64, 128, 2), (100, 7168, 256, 8), (250, 1472, 256, 8), (255, 128, 128, 8),
                                     (256, 2048, 256, 8)])
def test_one_tile_of_rows(T, H, E, k):
    """Batches of at most 256 tokens form the logits a way of their own; the same
    bits with a prepared weight."""
    cfg, d = inputs(T, H, E, k, seed=3 * T + H)
    got, ws = run(cfg, d, True, True)
    assert ws.status() == 0
    check(cfg, d, got, True, True)
    again, _ = run(cfg, d, True, True, W_split=moe.prepare_router(cfg, d["W"]))
    assert all(torch.equal(got[n], again[n]) for n in ("d_hidden", "dW_router"))


def test_many_experts_per_token():
    cfg, d = inputs(300, 256, 256, 32, seed=5, keep=8)
    check(cfg, d, run(cfg, d, True, False)[0], True, False)


def test_saturated_scores():
    """Scores within 1e-6 of 1 and of 0 keep the digits of their slope."""
    cfg, d = inputs(200, 512, seed=6)
    d["W"] *= 6
    d["idx"], _, d["counts"], _, _ = moe.route(cfg, d["hidden"], d["W"])
    check(cfg, d, run(cfg, d, True, True)[0], True, True)


def test_repeated_and_bad_expert_ids():
    """A repeated id adds up; an id outside the experts is skipped and flagged."""
    cfg, d = inputs(70, 256, seed=7)
    d["idx"][:, 3] = d["idx"][:, 2]
    got, ws = run(cfg, d, False, False)
    assert ws.status() == 0
    check(cfg, d, got, False, False)
    d["idx"][5, 1], d["idx"][6, 0], d["idx"][69, 7] = -1, 256, 1 << 30
    ok = (d["idx"] >= 0) & (d["idx"] < 256)
    got, ws = run(cfg, d, False, False)
    assert ws.status() == _lib.MOE_STATUS_BAD_EXPERT_INDEX
    check(cfg, d, got, False, False, idx_ok=ok)


def test_nonfinite_logits_are_flagged():
    cfg, d = inputs(70, 256, seed=8)
    d["hidden"][9] = float("nan")
    got, ws = run(cfg, d, False, False)
    assert ws.status() == _lib.MOE_STATUS_NONFINITE_LOGIT
    rows = [i for i in range(70) if i != 9]
    assert torch.isfinite(got["d_hidden"][rows].float()).all()


def test_split_given_in_place_and_streams():
    """A prepared weight, d_hidden over d_hidden_add and a side stream: the same bits."""
    cfg, d = inputs(600, 1024, seed=9)
    want, _ = run(cfg, d, True, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        over = d["add"].clone()
        got = moe.route_backward(cfg, d["hidden"], d["W"], d["idx"], d["d_w"], d_aux_loss=d["d_aux"],
                                 expert_counts=d["counts"], d_hidden_add=over,
                                 W_split=moe.prepare_router(cfg, d["W"]), out=dict(d_hidden=over))
    side.synchronize()
    assert got["d_hidden"] is over
    assert torch.equal(over, want["d_hidden"]) and torch.equal(got["dW_router"], want["dW_router"])


def test_differences():
    """Directional central differences of the kernels' own routing weights in 64
    bits, the choice of experts held fixed."""
    cfg, d = inputs(40, 128, seed=10)
    got, _ = run(cfg, d, True, False)

    def value(x, W):
        s = torch.sigmoid(x @ W.t())
        c = s.gather(1, d["idx"].long())
        w = c / (c.sum(1, keepdim=True) + cfg.eps) * cfg.rsf
        f = d["counts"].double() / (cfg.k * cfg.T)
        return (w * d["d_w"].double()).sum() + d["d_aux"].double()[0] * cfg.E * (f * (s / s.sum(1, keepdim=True)).mean(0)).sum()

    x, W = d["hidden"].double(), d["W"].double()
    for name, leaf in (("d_hidden", x), ("dW_router", W)):
        t = torch.randn(leaf.shape, generator=torch.Generator().manual_seed(3)).to(DEV).double()
        e = 1e-5
        a, b = (value(x + e * t, W), value(x - e * t, W)) if leaf is x else (value(x, W + e * t), value(x, W - e * t))
        want, have = ((a - b) / (2 * e)).item(), (got[name].double() * t).sum().item()
        slack = (2.0 ** -8 if leaf is x else 1e-4) * (got[name].double() * t).norm().item() * 4 + 1e-5
        assert abs(have - want) <= slack, (name, have, want)


@pytest.mark.parametrize("bad,error", [
    (dict(idx="long"), TypeError), (dict(d_w="half"), TypeError), (dict(W="short"), ValueError),
    (dict(add="float"), TypeError), (dict(counts="none"), _lib.MoeError),
])
def test_refusals(bad, error):
    cfg, d = inputs(16, 256)
    (name, how), = bad.items()
    t = d[name]
    d[name] = {"long": lambda: t.long(), "half": lambda: t.half(), "short": lambda: t[:128], "float": lambda: t.float(),
               "none": lambda: None}[how]()
    with pytest.raises(error):
        moe.route_backward(cfg, d["hidden"], d["W"], d["idx"], d["d_w"], d_aux_loss=d["d_aux"],
                           expert_counts=d["counts"], d_hidden_add=d["add"])
