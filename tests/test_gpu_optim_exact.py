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


def every_exponent(seed):
    """Values of every exponent, zero, the largest numbers, infinity and NaN."""
    rng = np.random.default_rng(seed)
    bits = (np.arange(255, dtype=np.uint32)[:, None] << 23) | rng.integers(0, 1 << 23, (255, 64), dtype=np.uint32)
    ends = np.array([0, 1, 2, 0x7fffff, 0x800000, 0x7f7fffff, 0x7f800000, 0x7fc00000], np.uint32)
    return np.concatenate([bits.ravel(), ends]).view(f)


@pytest.mark.parametrize("eps", [0.0, 1e-8])
def test_roots_of_every_size(eps):
    """No second moment is too large or too small for its root: an infinite one stops
    the parameter, a subnormal one moves it by lr."""
    v = every_exponent(1)
    n = v.size
    m = (np.where(np.isfinite(v) & (v > 0), np.sqrt(v), f(1)) * np.random.default_rng(2).uniform(0.5, 2, n)).astype(f)
    zero = np.zeros(n, f)
    got = stepped(zero, zero, m, v, 1.0, 0.5, 0.5, eps)[0]
    with np.errstate(all="ignore"):
        m, v = m * f(0.5), v * f(0.5)
        root = np.sqrt(v).astype(np.float64)
        want = -(m.astype(np.float64) / (root / math.sqrt(0.5) + eps)) / 0.5
    ends = ~np.isfinite(v) | (want == 0)
    assert np.array_equal(got[ends], want[ends].astype(f), equal_nan=True)
    # a rounding each of the root, 1 / sqrt(1 - beta2), their product, eps and the sum,
    # the quotient and twice the product with lr: eight halves of a step at most
    with np.errstate(all="ignore"):
        far = np.abs(got - want) / np.abs(want)
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf].astype(f))
    assert far[~ends & ~inf].max() <= 8 * 2.0 ** -24


def random_bits(n, key):
    x = (np.arange(n, dtype=np.uint64) * np.uint64(0x9E3779B9) + np.uint64(key)) & np.uint64(0xffffffff)
    for shift, times in ((16, 0x6A09E667), (15, 0xBB67AE85)):
        x ^= x >> np.uint64(shift)
        x = (x * np.uint64(times)) & np.uint64(0xffffffff)
    return x ^ (x >> np.uint64(16))


def key(seed, step, ordinal=0):
    return (seed + step * 0x85A308D3 + ordinal * 0x13198A2F) & 0xffffffff


def to_bytes(x, u, up):
    """x [n] fp32 -> (e4m3 values, scale bytes) by the rounding rule (the sum with the
    random fraction rounded to fp32, all else exact)."""
    n = x.size
    b = np.pad(x.astype(np.float64), (0, -n % 128)).reshape(-1, 128)
    top = np.abs(b).max(1)
    bad = ~np.isfinite(top)
    m, e = np.frexp(np.where(bad, 1.0, top) / 448.0)
    e = np.maximum(np.where(top > 0, np.where(m == 0.5, e - 1, e), 0), -127)
    t = np.abs(np.where(bad[:, None], 0.0, b)) / np.exp2(e.astype(np.float64))[:, None]
    step = np.exp2(np.maximum(np.frexp(t)[1] - 1, -6) - 3.0)
    fraction = np.pad(u.astype(np.float64), (0, -n % 128)).reshape(-1, 128) / 65536
    q = np.floor((t / step).astype(f) + fraction.astype(f)).astype(np.float64)
    if up:
        q = np.where((q == 0) & (t > 0), 1.0, q)
    q = np.where(bad[:, None], np.nan, np.sign(b) * q * step)
    return q.ravel()[:n], np.where(bad, 255, e + 127)


def check_bytes(opt, i, name, x, u, up):
    q, scale = to_bytes(x, u, up)
    assert np.array_equal(opt.state[name + "_scale"][i].view(torch.uint8).cpu().numpy(), scale)
    assert np.array_equal(host(opt.state[name][i]), q.astype(f), equal_nan=True)


def spread(opt, i, name):
    """The values that 8-bit states stand for (exact in fp32 but for the smallest)."""
    q, s = opt.state[name][i].double(), opt.state[name + "_scale"][i].double()
    return (q * s.repeat_interleave(128)[:q.numel()]).cpu().numpy().astype(f)


@pytest.mark.parametrize("lo,hi", [(-20, 0), (60, 66), (80, 100)])
def test_large_roots_in_8_bits(lo, hi):
    """The root of a square past fp32's range is infinite, and so its block's scale NaN."""
    n, b1, b2 = 4000, 0.9, 0.999
    g = gradient_sizes(n, 3, lo, hi)
    zero = np.zeros(n, f)
    p = on(zero)
    opt = optim.AdamW([p], lr=1e-3, betas=(b1, b2), weight_decay=0.0, state_bits=8, seed=5)
    opt.step([on(g)])
    want, m, v, root = formula(zero, g, zero, zero, 1, 1e-3, b1, b2, 1e-8, 0.0)
    bits = random_bits(n, key(5, 1))
    check_bytes(opt, 0, "m", m, bits & np.uint64(0xffff), False)
    check_bytes(opt, 0, "v", root, bits >> np.uint64(16), True)
    assert np.abs(host(p) - want).max() <= 2.0 ** -20 * np.abs(want).max()


@pytest.mark.parametrize("lr,b1,b2,eps,decay", [(1e-3, 0.9, 0.999, 1e-8, 0.1), (0.3, 0.8, 0.95, 1e-15, 0.0),
                                                (1e-3, 0.0, 0.5, 0.0, 0.1), (1e-25, 0.9, 0.99, 1e-30, 0.1)])
@pytest.mark.parametrize("lo,hi", [(-16, 0), (-45, 70)])
def test_a_step_is_the_formula_to_the_bit(lo, hi, lr, b1, b2, eps, decay):
    n = 200003
    p, g = gradient_sizes(n, 4, -6, 0), gradient_sizes(n, 5, lo, hi)
    m, v = gradient_sizes(n, 6, lo, hi), np.square(gradient_sizes(n, 7, max(lo, -40), hi / 2))
    p[:300], g[128:512], m[256:900], v[384:700] = 0, 0, 0, 0
    got = stepped(p, g, m, v, lr, b1, b2, eps, decay, step=6)
    want = formula(p, g, m, v, 7, lr, b1, b2, eps, decay)
    for a, b in zip(got, want):
        assert np.array_equal(a, b, equal_nan=True)


def test_every_mantissa():
    """All roots of a binade pair, and all quotients by them with some numerators:
    those of 1 are the reciprocals, on which the other quotients' rounding rests."""
    v = np.arange(1 << 24, dtype=np.uint32) + np.uint32(0x40000000)      # 2 to 8, halved by the step
    v = v.view(f)
    zero = np.zeros(v.size, f)
    rng = np.random.default_rng(8)
    for m in (np.full(v.size, 2, f), (rng.standard_normal(v.size) * np.exp2(rng.uniform(-30, 8, v.size))).astype(f)):
        got = stepped(zero, zero, m, v, 1.0, 0.5, 0.5, 1e-15, step=10 ** 6)     # 1 - beta^t is 1
        want = formula(zero, zero, m, v, 10 ** 6 + 1, 1.0, 0.5, 0.5, 1e-15, 0.0)
        assert np.array_equal(got[0], want[0])
    # many numerators over the divisors next to a power of two
    roots = np.concatenate([np.nextafter(f(2), f(0), dtype=f) - np.arange(8, dtype=f) * f(2.0 ** -23),
                            f(1) + np.arange(8, dtype=f) * f(2.0 ** -23)])
    v = np.square(roots.astype(np.float64)).astype(f)
    keep = np.sqrt(v) == roots
    assert keep.sum() >= 8
    v = (v[keep] * f(2)).repeat(1 << 16)
    m = rng.uniform(2, 4, v.size).astype(f)
    zero = np.zeros(v.size, f)
    got = stepped(zero, zero, m, v, 1.0, 0.5, 0.5, 1e-15, step=10 ** 6)
    want = formula(zero, zero, m, v, 10 ** 6 + 1, 1.0, 0.5, 0.5, 1e-15, 0.0)
    assert np.array_equal(got[0], want[0])


@pytest.mark.parametrize("grad", [BF, F32])
@pytest.mark.parametrize("param,master", [(BF, False), (BF, True), (F32, False)])
@pytest.mark.parametrize("lo,hi", [(-16, 0), (-60, 66)])
def test_8_bit_steps_are_the_formula_to_the_bit(lo, hi, param, master, grad):
    """Values in 8 bits and stochastically rounded parameters included: an ulp in fp32
    would put some of them on the other side of a rounding's border."""
    sizes = [1, 127, 128, 129, 513, 4097, 300001]
    params = [on(gradient_sizes(n, 10 + n, -6, 0)).to(param) for n in sizes]
    lr, b1, b2, eps, decay, seed = 1e-2, 0.9, 0.99, 1e-8, 0.1, 987654321
    opt = optim.AdamW(params, lr=lr, betas=(b1, b2), eps=eps, weight_decay=decay, state_bits=8, master=master, seed=seed)
    for t in (1, 2, 3):
        grads = [on(gradient_sizes(n, 20 + t, lo, hi)).to(grad) for n in sizes]
        for g in grads:
            g[100:400] = 0
        old = [(host(opt.state["master"][i] if master else p), spread(opt, i, "m"), spread(opt, i, "v"))
               for i, p in enumerate(params)]
        opt.step(grads)
        for i, (w, m, root) in enumerate(old):
            n = sizes[i]
            want, m, v, root = formula(w, host(grads[i]), m, np.square(root), t, lr, b1, b2, eps, decay)
            bits = random_bits(n, key(seed, t, i))
            check_bytes(opt, i, "m", m, bits & np.uint64(0xffff), False)
            check_bytes(opt, i, "v", root, bits >> np.uint64(16), True)
            if param == F32 or master:
                assert np.array_equal(host(opt.state["master"][i] if master else params[i]), want, equal_nan=True)
                assert not master or np.array_equal(host(params[i]), host(opt.state["master"][i].to(BF)), equal_nan=True)
                continue
            u = (((bits * np.uint64(0x9E3779B9)) & np.uint64(0xffffffff)) >> np.uint64(16)).astype(np.int32)
            rounded = ((want.view(np.int32) + u) & np.int32(-65536)).view(f)
            assert np.array_equal(host(params[i]), np.where(np.isnan(want), want, rounded), equal_nan=True)


@pytest.mark.parametrize("exponent", [-150, -136, -128, -120, -90])
def test_the_smallest_states_in_8_bits(exponent):
    """Scales down to the format's smallest, 2^-127, where fp32 is subnormal."""
    n, b1, b2, seed = 1000, 0.9, 0.99, 3
    zero = np.zeros(n, f)
    p = on(zero)
    opt = optim.AdamW([p], lr=1e-3, betas=(b1, b2), eps=1e-8, weight_decay=0.0, state_bits=8, seed=seed)
    rng = np.random.default_rng(9)
    for name in ("m", "v"):
        opt.state[name + "_scale"][0].view(torch.uint8).copy_(on(np.full(-(-n // 128), max(0, 127 + exponent // (1 + (name == "v"))), np.uint8)))
        opt.state[name][0].view(torch.uint8).copy_(on(rng.integers(1, 127, n, dtype=np.uint8)))
    m, root = spread(opt, 0, "m"), spread(opt, 0, "v")
    opt.step([on(zero)])
    want, m, v, root = formula(zero, zero, m, np.square(root), 1, 1e-3, b1, b2, 1e-8, 0.0)
    bits = random_bits(n, key(seed, 1))
    check_bytes(opt, 0, "m", m, bits & np.uint64(0xffff), False)
    check_bytes(opt, 0, "v", root, bits >> np.uint64(16), True)


def test_the_largest_first_moments_in_8_bits():
    """A block's largest magnitude between 1.75 2^127 and fp32's largest number is no
    infinity: its scale is 2^120."""
    n, seed = 128 * 4, 3
    g = np.full(n, 2.0 ** 100, f)
    g[5], g[130], g[300], g[400] = MAX, -f(1.75 * 2.0 ** 127), np.nextafter(f(1.75 * 2.0 ** 127), f(np.inf)), np.inf
    p = torch.zeros(n, device=DEV)
    opt = optim.AdamW([p], lr=0.0, betas=(0.0, 0.9), weight_decay=0.0, state_bits=8, seed=seed)
    opt.step([on(g)])
    check_bytes(opt, 0, "m", g, random_bits(n, key(seed, 1)) & np.uint64(0xffff), False)
    assert opt.state["m_scale"][0].view(torch.uint8).tolist() == [247, 246, 247, 255]
