"""block_norm and its gradient on the GPU against the formulas in 64 bits.

Tolerances, element by element, from the arithmetic: a bf16 output is rounded
by at most half a step, 2^-8 of its value; everything before that is fp32, and
each quantity is a short chain of roundings of the magnitudes it is summed
from (a row sum is at most 16 additions per thread, 5 across a warp and 16
across warps, so 64 half-steps of 2^-24 cover r and n, and 128 the gradients'
longer chains); a column sum adds up to 27 rows in a block, then up to 76
blocks, then 32 partial sums, so 256."""
import pytest
import torch

from group_limited_routing_gb300 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24


def inputs(T, H, groups, stream, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(x=(rnd(T, H) * 2 * scale).to(stream), y=(rnd(T, H) * 0.3 * scale).bfloat16(),
             gate=None if groups is None else rnd(groups, H) * 0.2 + 0.5, w_post=rnd(H) * 0.1 + 1,
             w_pre=rnd(H) * 0.1 + 1, d_r=rnd(T, H).to(stream), d_n=rnd(T, H).bfloat16())
    return {k: None if v is None else v.to(DEV) for k, v in d.items()}


def formulas(d, alpha, eps, has_y=True):
    """Everything in 64 bits, and the magnitudes the outputs are summed from."""
    f = {k: None if v is None else v.double() for k, v in d.items()}
    T, H = f["x"].shape
    one = torch.ones(H, dtype=torch.float64, device=DEV)
    pre = one if f["w_pre"] is None else f["w_pre"]
    post = one if f["w_post"] is None else f["w_post"]
    gate = one[None] if f["gate"] is None else f["gate"]
    G = gate.shape[0]
    rows = gate.repeat_interleave(T // G, 0)
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    ax = alpha * f["x"]
    o, m = {}, {}
    if has_y:
        rho = 1 / (mean(f["y"] ** 2) + eps).sqrt()
        u = f["y"] * rho
        v = rows * post * u
    else:
        u = v = torch.zeros_like(ax)
    r = ax + v
    m["r"] = ax.abs() + v.abs()
    sigma = 1 / (mean(r ** 2) + eps).sqrt()
    q = r * sigma
    o["r"], o["n"] = r, q * pre
    m["n"] = m["r"] * sigma * pre.abs()
    mq = m["r"] * sigma
    dq = f["d_n"] * pre
    d_r = torch.zeros_like(ax) if f["d_r"] is None else f["d_r"]
    dr = d_r + sigma * (dq - q * mean(dq * q))
    mdr = d_r.abs() + sigma * (dq.abs() + mq * mean(dq.abs() * mq))
    o["d_x"], m["d_x"] = alpha * dr, abs(alpha) * mdr
    o["dw_pre"], m["dw_pre"] = (f["d_n"] * q).sum(0), (f["d_n"].abs() * mq).sum(0)
    if has_y:
        du, mdu = dr * rows * post, mdr * (rows * post).abs()
        o["d_y"] = rho * (du - u * mean(du * u))
        m["d_y"] = rho * (mdu + u.abs() * mean(mdu * u.abs()))
        fold = lambda t: t.view(G, -1, H).sum(1)  # noqa: E731
        o["d_gate"], m["d_gate"] = fold(dr * post * u), fold(mdr * (post * u).abs())
        o["dw_post"], m["dw_post"] = (dr * rows * u).sum(0), (mdr * (rows * u).abs()).sum(0)
    return o, m


STEPS = dict(r=64, n=64, d_x=128, d_y=128, d_gate=256, dw_post=256, dw_pre=256)


def check(got, d, alpha, eps, has_y=True):
    o, m = formulas(d, alpha, eps, has_y)
    for name, t in got.items():
        assert t.shape == o[name].shape, name
        bound = HALF[t.dtype] * o[name].abs() + STEPS[name] * U * m[name] + 1e-37
        over = ((t.double() - o[name]).abs() / bound).max().item()
        assert over <= 1.0, "%s off by %.3g of its bound" % (name, over)


def run(d, alpha=0.9, eps=1e-6):
    r, n = moe.block_norm(d["x"], d["y"], d["gate"], d["w_post"], d["w_pre"], alpha=alpha, eps=eps)
    check(dict(r=r, n=n), d, alpha, eps, d["y"] is not None)
    g = moe.block_norm_backward(d["x"], d["y"], d["gate"], d["w_post"], d["w_pre"], d["d_r"], d["d_n"], alpha=alpha,
                                eps=eps)
    check(g, d, alpha, eps, d["y"] is not None)
    return r, n, g


@pytest.mark.parametrize("T,H,groups", [
    (1, 8, 1), (1, 2048, 1), (2, 264, 2), (3, 1000, None), (16, 2048, 1), (16, 2048, 16), (33, 4096, 1),
    (130, 512, 5), (257, 2056, 1), (700, 1536, 7), (1021, 256, 1), (95, 8192, 5), (4100, 2048, 2050), (5000, 520, 40),
])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_formulas(T, H, groups, stream):
    run(inputs(T, H, groups, stream, seed=T + H))


@pytest.mark.parametrize("drop", [("gate",), ("w_post", "w_pre"), ("d_r",), ("gate", "w_post", "w_pre", "d_r")])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_absent_parts(drop, stream):
    d = inputs(70, 1032, 7, stream, seed=5)
    run({k: None if k in drop else v for k, v in d.items()})


@pytest.mark.parametrize("H", [64, 2048, 6000])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_without_a_block(H, stream):
    d = inputs(77, H, None, stream, seed=9)
    d.update(y=None, w_post=None)
    r, n, g = run(d, alpha=1.0)
    assert torch.equal(r, d["x"]) and set(g) == {"d_x", "dw_pre"}


def test_zero_rows_and_eps():
    """Rows of zeros: 1 / sqrt(eps) scales nothing, no NaN; eps = 0 elsewhere."""
    d = inputs(40, 512, 4, torch.bfloat16, seed=3)
    for name in ("x", "y"):
        d[name][3] = 0
        d[name][39] = 0
    r, n, g = run(d)
    assert not n[3].any() and not r[39].any()
    run(inputs(40, 512, 4, torch.bfloat16, seed=4), eps=0.0)


def test_nonfinite_rows_stay_in_their_rows():
    d = inputs(20, 256, 4, torch.bfloat16, seed=8)
    clean = moe.block_norm(d["x"], d["y"], d["gate"], d["w_post"], d["w_pre"])
    d["y"][5, 7] = float("nan")
    d["x"][6, 0] = float("inf")
    r, n = moe.block_norm(d["x"], d["y"], d["gate"], d["w_post"], d["w_pre"])
    assert torch.isnan(n[5]).all() and torch.isnan(n[6, 0])
    keep = [i for i in range(20) if i not in (5, 6)]
    assert torch.equal(r[keep], clean[0][keep]) and torch.equal(n[keep], clean[1][keep])


def test_in_place_streams_and_repeats():
    """r over x and n over y, gradients over their inputs, on a side stream; the
    same bits every time."""
    d = inputs(1000, 2048, 4, torch.bfloat16, seed=11)
    a = (d["x"], d["y"], d["gate"], d["w_post"], d["w_pre"])
    r, n = moe.block_norm(*a)
    g = moe.block_norm_backward(*a, d["d_r"], d["d_n"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x, y, d_r, d_n = (d[k].clone() for k in ("x", "y", "d_r", "d_n"))
        g2 = moe.block_norm_backward(x, y, *a[2:], d_r, d_n, out=dict(d_x=d_r, d_y=d_n))
        r2, n2 = moe.block_norm(x, y, *a[2:], out=(x, y))
    side.synchronize()
    assert r2 is x and torch.equal(r2, r) and torch.equal(n2, n)
    for name in g:
        assert torch.equal(g2[name], g[name]), name


def test_differences():
    """The gradient against central differences of the forward, along random
    directions of every leaf (fp32 stream; the forward's n is bf16, so the
    differences are taken of the 64-bit formula, pinned to the kernel above)."""
    d = inputs(24, 128, 3, torch.float32, seed=21)
    g = moe.block_norm_backward(d["x"], d["y"], d["gate"], d["w_post"], d["w_pre"], d["d_r"], d["d_n"], alpha=0.8)

    def value(e):
        o, _ = formulas(e, 0.8, 1e-6)
        return (o["r"] * d["d_r"].double()).sum() + (o["n"] * d["d_n"].double()).sum()

    names = dict(x="d_x", y="d_y", gate="d_gate", w_post="dw_post", w_pre="dw_pre")
    for leaf, grad in names.items():
        t = torch.randn(d[leaf].shape, generator=torch.Generator().manual_seed(1)).to(DEV).double()
        h = 1e-4
        plus = value({**{k: v.double() for k, v in d.items()}, leaf: d[leaf].double() + h * t})
        minus = value({**{k: v.double() for k, v in d.items()}, leaf: d[leaf].double() - h * t})
        want = ((plus - minus) / (2 * h)).item()
        got = (g[grad].double() * t).sum().item()
        # each element rounded by half a step at most, h^2 of the differences
        slack = (HALF[g[grad].dtype] * g[grad].double().abs() * t.abs()).sum().item() + 1e-3
        assert abs(got - want) <= slack, (leaf, got, want)


@pytest.mark.parametrize("bad,error", [
    (dict(y="cpu"), ValueError), (dict(y="wide"), ValueError), (dict(x="half"), TypeError), (dict(gate="bf16"), TypeError),
    (dict(w_pre="short"), ValueError), (dict(y="strided"), ValueError), (dict(gate="3rows"), moe._lib.MoeError),
])
def test_refusals(bad, error):
    d = inputs(16, 256, 4, torch.bfloat16)
    (name, how), = bad.items()
    t = d[name]
    d[name] = {"cpu": lambda: t.cpu(), "wide": lambda: torch.cat([t, t], 1), "half": lambda: t.half(),
               "bf16": lambda: t.bfloat16(), "short": lambda: t[:128], "strided": lambda: torch.cat([t, t], 1)[:, ::2],
               "3rows": lambda: t[:3]}[how]()
    with pytest.raises(error):
        moe.block_norm(d["x"], d["y"], d["gate"], d["w_post"], d["w_pre"])
