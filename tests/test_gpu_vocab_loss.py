"""vocab_loss and its gradient on the GPU against the formulas in 64 bits.

Tolerances, element by element, from the arithmetic.  A logit is a sum of exact
products in steps of 16 on the tensor core, each step off by at most one unit
in the last place (2^-23) of the magnitudes summed.  lse: the exponentials' and
sums' errors are below 128 half-steps of 2^-24 (two chains of 32 per 64
columns, four of those per tile, tiles / 32 per warp, 32 warps), the
exponents' roundings below 2^-24 of 4 |z| and of 4 |lse|.  Gradient: dz is
rounded to bf16 (half a step, 2^-8), the products add in fp32, the result is
rounded to bf16 once more.  Over a whole gradient the independent roundings of
dz and of the result stay below 2^-8 each in the 2-norm."""
import pytest
import torch

from group_limited_routing_gb300 import _lib, moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
IGN = -100


def inputs(T, H, V, ignored=0.0, seed=0, lean=8.0, bits=torch.int64):
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn(V, H, generator=g) * (0.9 / H ** 0.5)).bfloat16()
    target = torch.randint(0, V, (T,), generator=g)
    pull = torch.rand(T, 1, generator=g) * lean / 0.81
    hidden = (torch.randn(T, H, generator=g) + pull * W[target].float()).bfloat16()
    target[torch.rand(T, generator=g) < ignored] = IGN
    d_loss = (torch.rand(T, generator=g) + 0.5) / max(T, 1)
    return dict(hidden=hidden.to(DEV), W=W.to(DEV), target=target.to(bits).to(DEV), d_loss=d_loss.to(DEV))


def logits(d):
    h, W = d["hidden"].double(), d["W"].double()
    z = h @ W.t()
    zb = (h.shape[1] / 16 + 4) * 2 * U * (h.abs() @ W.abs().t())
    return z, zb


def keep_of(d, ignore=IGN):
    t, V = d["target"].long(), d["W"].shape[0]
    return (t != ignore) & (t >= 0) & (t < V)


def check_forward(d, loss, lse, ignore=IGN):
    keep = keep_of(d, ignore)
    assert not loss[~keep].any() and not lse[~keep].any()
    if not keep.any():
        return
    z, zb = logits(d)
    z, zb, t = z[keep], zb[keep], d["target"][keep].long()[:, None]
    ref = torch.logsumexp(z, 1)
    at, atb = z.gather(1, t)[:, 0], zb.gather(1, t)[:, 0]
    bound = zb.amax(1) + U * (128 + 4 * z.abs().amax(1) + 4 * ref.abs())
    over = ((lse[keep].double() - ref).abs() / bound).max().item()
    assert over <= 1, "lse off by %.3g of its bound" % over
    over = ((loss[keep].double() - (ref - at)).abs() / (bound + atb + U * (at.abs() + ref.abs()))).max().item()
    assert over <= 1, "loss off by %.3g of its bound" % over


def check_backward(d, lse, got, ignore=IGN):
    keep = keep_of(d, ignore)
    assert not got["d_hidden"][~keep].any()
    if not keep.any():
        assert not got["dW_vocab"].any()
        return
    z, zb = logits(d)
    z, zb, l = z[keep], zb[keep], lse[keep].double()[:, None]
    g = d["d_loss"][keep].double()[:, None]
    h, W = d["hidden"][keep].double(), d["W"].double()
    p = (z - l).exp()
    dz = g * (p - torch.zeros_like(p).scatter_(1, d["target"][keep].long()[:, None], 1.0))
    plain = g.abs() * p * (zb + U * (8 + 4 * z.abs() + 4 * l.abs()))       # fp32 errors of p, which p - 1 may leave alone
    err = dz.abs() * (2.0 ** -8 + 4 * U) + plain
    steps = 2 * U * (max(p.shape) / 16 + 24)
    for name, ref, bound, rest in (
            ("d_hidden", dz @ W, err @ W.abs() + steps * (dz.abs() @ W.abs()), plain @ W.abs()),
            ("dW_vocab", dz.t() @ h, err.t() @ h.abs() + steps * (dz.abs().t() @ h.abs()), plain.t() @ h.abs())):
        out = (got[name][keep] if name == "d_hidden" else got[name]).double()
        bound = bound + 2.0 ** -8 * ref.abs() + 1e-37
        over = ((out - ref).abs() / bound).max().item()
        assert over <= 1, "%s off by %.3g of its bound" % (name, over)
        far = ((out - ref).norm() / (2 * 2.0 ** -8 * ref.norm() + rest.norm() + 1e-37)).item()
        assert far <= 1, "%s off by %.3g of its bound in the 2-norm" % (name, far)


def run(d, ignore=IGN):
    T, H = d["hidden"].shape
    ws = moe.vocab_loss_workspace(T, H, d["W"].shape[0])
    loss, lse = moe.vocab_loss(d["hidden"], d["W"], d["target"], ignore_index=ignore, ws=ws)
    check_forward(d, loss, lse, ignore)
    wb = moe.vocab_loss_workspace(T, H, d["W"].shape[0], backward=True)
    g = moe.vocab_loss_backward(d["hidden"], d["W"], d["target"], lse, d["d_loss"], ignore_index=ignore, ws=wb)
    check_backward(d, lse, g, ignore)
    return loss, lse, g, ws.status() | wb.status()


@pytest.mark.parametrize("T,H,V,ignored", [
    (1, 8, 1, 0.0), (1, 64, 2, 0.0), (2, 72, 255, 0.0), (3, 128, 256, 0.0), (5, 136, 257, 0.0), (127, 512, 1000, 0.0),
    (129, 264, 3001, 0.3), (255, 520, 777, 0.0), (256, 256, 512, 0.5), (257, 2056, 640, 0.0), (1, 2048, 20000, 0.0),
    (600, 64, 5003, 0.9), (1030, 320, 2050, 0.1), (64, 4096, 1031, 0.0),
])
def test_formulas(T, H, V, ignored):
    *_, status = run(inputs(T, H, V, ignored, seed=T + V))
    assert status == 0


def test_int32_targets_and_an_ignored_id_inside_the_vocabulary():
    d = inputs(200, 128, 50, seed=1, bits=torch.int32)
    *_, status = run(d, ignore=7)
    assert status == 0


@pytest.mark.parametrize("rows", [0, 1, 63, 64, 65, 300])
def test_rows_that_count(rows):
    """None, one, and numbers around a K block, scattered among ignored rows
    whose hidden states are NaN and infinite."""
    d = inputs(300, 96, 700, seed=rows)
    masked = torch.randperm(300, generator=torch.Generator().manual_seed(5))[rows:].to(DEV)
    d["target"][masked] = IGN
    clean = d["hidden"].clone()
    d["hidden"][masked[::2]] = float("nan")
    d["hidden"][masked[1::2]] = float("inf")
    d["d_loss"][masked] = float("nan")
    loss, lse = moe.vocab_loss(d["hidden"], d["W"], d["target"])
    g = moe.vocab_loss_backward(d["hidden"], d["W"], d["target"], lse, d["d_loss"])
    d["hidden"] = clean
    check_forward(d, loss, lse)
    check_backward(d, lse, g)


def test_targets_out_of_range_are_flagged_and_skipped():
    d = inputs(90, 64, 100, seed=2)
    for i, v in enumerate((100, -1, 1 << 40, -(1 << 62), 2147483647)):
        d["target"][7 * i] = v
    loss, lse, g, status = run(d)
    assert status == _lib.MOE_STATUS_BAD_TARGET
    assert not loss[0] and not g["d_hidden"][0].any()


def test_no_rows():
    d = inputs(0, 64, 100)
    loss, lse = moe.vocab_loss(d["hidden"], d["W"], d["target"])
    g = moe.vocab_loss_backward(d["hidden"], d["W"], d["target"], lse, d["d_loss"])
    assert loss.shape == (0,) and g["d_hidden"].shape == (0, 64) and not g["dW_vocab"].any()


@pytest.mark.parametrize("scale", [30.0, 3000.0])
def test_large_logits(scale):
    """Logits of several hundred and of tens of thousands: no overflow, and
    rows whose softmax is a single column."""
    d = inputs(140, 256, 900, seed=4)
    d["hidden"] = (d["hidden"].float() * scale).bfloat16()
    run(d)


def test_equal_logits_and_a_zero_gradient():
    d = inputs(40, 64, 1000, seed=6)
    d["hidden"].zero_()
    loss, lse, g, _ = run(d)
    d["d_loss"].zero_()
    g = moe.vocab_loss_backward(d["hidden"], d["W"], d["target"], lse, d["d_loss"])
    assert not g["d_hidden"].any() and not g["dW_vocab"].any()


def test_infinite_and_nan_logits_show_in_their_rows_only():
    d = inputs(20, 64, 300, seed=7)
    clean, _ = moe.vocab_loss(d["hidden"], d["W"], d["target"])
    d["hidden"][3] = float("nan")
    d["hidden"][4, 0] = float("inf")
    d["W"][:, 0] = d["W"][:, 0].abs() + 0.01           # row 4: every logit +inf
    base, _ = moe.vocab_loss(torch.where(d["hidden"].isfinite(), d["hidden"], 0.0), d["W"], d["target"])
    loss, lse = moe.vocab_loss(d["hidden"], d["W"], d["target"])
    assert torch.isnan(loss[3]) and torch.isnan(lse[3])
    assert lse[4] == float("inf") and torch.isnan(loss[4])
    keep = [i for i in range(20) if i not in (3, 4)]
    assert torch.equal(loss[keep], base[keep]) and torch.isfinite(clean).all()


@pytest.mark.parametrize("T,H,V,keep", [(1, 64, 300, 1), (3, 1000, 5000, 3), (16, 512, 1111, 16), (17, 72, 600, 17),
                                        (31, 1544, 3000, 31), (32, 256, 2000, 32), (33, 256, 2000, 32),
                                        (40, 128, 700, 9), (150, 128, 700, 0), (1000, 264, 900, 31)])
def test_few_rows_gradient_keeps_its_digits(T, H, V, keep):
    """Up to 32 rows that count, dz is two bf16 parts: what is left out of it is
    half a step of half a step, 2^-16, so that only the result's rounding, 2^-8,
    is of bf16's size."""
    d = inputs(T, H, V, seed=T + V)
    off = torch.randperm(T, generator=torch.Generator().manual_seed(T))[keep:]
    d["target"][off.to(DEV)] = IGN
    _, lse, g, status = run(d)
    assert status == 0
    k = keep_of(d)
    if keep == 0:
        return                      # (check_backward: zeros)
    z, zb = logits(d)
    z, zb, l = z[k], zb[k], lse[k].double()[:, None]
    h, W, t = d["hidden"][k].double(), d["W"].double(), d["target"][k].long()[:, None]
    p = (z - l).exp()
    w = d["d_loss"][k].double()[:, None]
    dz = w * (p - torch.zeros_like(p).scatter_(1, t, 1.0))
    err = dz.abs() * (2.0 ** -16 + 4 * U) + w * p * (zb + U * (8 + 4 * z.abs() + 4 * l.abs()))
    steps = 2 * U * (max(p.shape) / 16 + 24)
    for name, ref, bound in (("d_hidden", dz @ W, err @ W.abs() + steps * (dz.abs() @ W.abs())),
                             ("dW_vocab", dz.t() @ h, err.t() @ h.abs() + steps * (dz.abs().t() @ h.abs()))):
        out = (g[name][k] if name == "d_hidden" else g[name]).double()
        over = ((out - ref).abs() / (bound + 2.0 ** -8 * ref.abs() + 1e-37)).max().item()
        assert over <= 1, "%s off by %.3g of its bound" % (name, over)


def test_several_vocabulary_pieces():
    """dz of the whole vocabulary would pass the workspace's piece."""
    d = inputs(4096, 64, 140001, ignored=0.02, seed=8)
    *_, status = run(d)
    assert status == 0


def test_a_long_batch():
    run(inputs(9000, 72, 1500, ignored=0.1, seed=12))


def test_repeats_and_streams_and_graphs():
    """The same bits on a side stream, and from a graph replayed on new inputs;
    a workspace used for one shape after another."""
    d, e = inputs(333, 256, 4000, 0.2, seed=9), inputs(333, 256, 4000, 0.6, seed=10)
    small = inputs(7, 64, 50, 0.0, seed=11)
    ws, wb = moe.vocab_loss_workspace(333, 256, 4000), moe.vocab_loss_workspace(333, 256, 4000, backward=True)

    def step(i):
        loss, lse = moe.vocab_loss(i["hidden"], i["W"], i["target"], ws=ws)
        g = moe.vocab_loss_backward(i["hidden"], i["W"], i["target"], lse, i["d_loss"], ws=wb)
        return loss, lse, g["d_hidden"], g["dW_vocab"]

    want_d, want_e = [t.clone() for t in step(d)], [t.clone() for t in step(e)]
    check_forward(e, *want_e[:2])
    step(small)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step(d)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, want_d))
    static = {k: v.clone() for k, v in d.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(static)
    for src, want in ((e, want_e), (d, want_d)):
        for k, v in src.items():
            static[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert ws.status() == 0 and wb.status() == 0


def test_gradient_against_differences():
    """Directional central differences of the 64-bit loss at the same inputs."""
    d = inputs(48, 64, 500, ignored=0.2, seed=13)
    loss, lse, g, _ = run(d)
    keep = keep_of(d)
    w = torch.where(keep, d["d_loss"], 0.0).double()

    def value(h, W):
        z = h @ W.t()
        at = z.gather(1, d["target"].long().clamp(min=0)[:, None])[:, 0]
        return (w * (torch.logsumexp(z, 1) - at))[keep].sum()

    h, W = d["hidden"].double(), d["W"].double()
    for name, leaf in (("d_hidden", h), ("dW_vocab", W)):
        t = torch.randn(leaf.shape, generator=torch.Generator().manual_seed(3)).to(DEV).double()
        e = 1e-5
        a, b = (value(h + e * t, W), value(h - e * t, W)) if leaf is h else (value(h, W + e * t), value(h, W - e * t))
        want, got = ((a - b) / (2 * e)).item(), (g[name].double() * t).sum().item()
        # roundings of the gradient's elements and of dz, in the 2-norm, times the direction's length
        slack = 2 * 2.0 ** -8 * (g[name].double() * t).norm().item() * 4 + 1e-6
        assert abs(got - want) <= slack, (name, got, want, slack)


@pytest.mark.parametrize("bad,error", [
    (dict(target="int16"), TypeError), (dict(target="short"), ValueError), (dict(hidden="float"), TypeError),
    (dict(W="narrow"), ValueError), (dict(hidden="strided"), ValueError), (dict(W="cpu"), ValueError),
    (dict(target="cpu"), ValueError), (dict(both="odd"), _lib.MoeError), (dict(hidden="flat"), TypeError),
])
def test_refusals(bad, error):
    d = inputs(16, 64, 100)
    (name, how), = bad.items()
    if how == "odd":
        d["hidden"], d["W"] = d["hidden"][:, :60].contiguous(), d["W"][:, :60].contiguous()
    else:
        t = d[name]
        d[name] = {"int16": lambda: t.short(), "short": lambda: t[:5], "float": lambda: t.float(), "cpu": lambda: t.cpu(),
                   "narrow": lambda: t[:, :32].contiguous(), "flat": lambda: t.flatten(),
                   "strided": lambda: torch.cat([t, t], 1)[:, ::2]}[how]()
    with pytest.raises(error):
        moe.vocab_loss(d["hidden"], d["W"], d["target"])
    with pytest.raises(error):
        moe.vocab_loss_backward(d["hidden"], d["W"], d["target"], d["d_loss"], d["d_loss"])
