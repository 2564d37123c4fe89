"""The pre-norm stack (MoEStack: x + layer(RMS x) for every layer) differentiated with
the library's calls: block_norm without a block output is its norm, and
block_norm_backward takes the stream's gradient as d_r, the layer's as d_n.

Tolerance, as in test_gpu_train: some 15 bf16 roundings a layer lie between the
stream and a gradient, each 2^-8 of its value at most and independent, so
sqrt(15 L) 2^-8 in the 2-norm."""
import pytest
import torch

from group_limited_routing_gb300 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_gradients_of_a_pre_norm_stack():
    T, H, I, L, eps = 96, 512, 256, 2, 1e-6
    g = torch.Generator().manual_seed(11)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    cfg = moe.MoeConfig(T=T, H=H, I=I, Is=I)
    bf = lambda *s: (rnd(*s) * 0.04).bfloat16().to(DEV)  # noqa: E731
    layers = [moe.MoELayer(cfg, (rnd(cfg.E, H) * 0.04).to(DEV), None, bf(cfg.E, 2 * I, H), bf(cfg.E, I, H),
                           bf(2 * I, H), bf(I, H)) for _ in range(L)]
    x, d_out = rnd(T, H).bfloat16().to(DEV), rnd(T, H).bfloat16().to(DEV)

    r, calls = x, []
    for layer in layers:
        n = moe.block_norm(r, eps=eps)[1]
        assert torch.equal(n, moe.rmsnorm(r, eps))
        calls.append((r, n))
        r = layer(n, residual=r)
    assert torch.equal(r, moe.MoEStack(layers, eps)(x))
    d, got = d_out, [None] * L
    for i in reversed(range(L)):
        layer, (r_in, n) = layers[i], calls[i]
        layer(n, residual=r_in)
        e = layer.backward(d)
        e.update(moe.route_backward(cfg, n, layer.W_router, layer.routing[0], e["d_topk_w"],
                                    d_hidden_add=e["d_hidden"]))
        d = moe.block_norm_backward(r_in, None, None, None, None, d, e["d_hidden"], eps=eps)["d_x"]
        got[i] = e

    f64 = lambda t: t.double().requires_grad_()  # noqa: E731
    names = ("W_router", "W_gate_up", "W_down", "shared_gate_up", "shared_down")
    leaves = [{k: f64(getattr(layer, k)) for k in names} for layer in layers]
    swiglu = lambda n, gu, down: (torch.nn.functional.silu(n @ gu[:I].t()) * (n @ gu[I:].t())) @ down  # noqa: E731
    first = s = f64(x)
    for layer, w in zip(layers, leaves):
        n = s / (s.pow(2).mean(1, keepdim=True) + eps).sqrt()
        idx = layer.routing[0].long()
        c = torch.sigmoid(n @ w["W_router"].t()).gather(1, idx)
        weight = c / (c.sum(1, keepdim=True) + cfg.eps) * cfg.rsf
        y = swiglu(n, w["shared_gate_up"], w["shared_down"])
        for e in range(cfg.E):
            t, j = (idx == e).nonzero(as_tuple=True)
            if t.numel():
                y = y.index_add(0, t, weight[t, j, None] * swiglu(n[t], w["W_gate_up"][e], w["W_down"][e]))
        s = s + y
    want = torch.autograd.grad((s * d_out.double()).sum(), [first] + [t for w in leaves for t in w.values()])
    pairs = [("d_x", d, want[0])]
    for i in range(L):
        for k, name in enumerate(("dW_router", "dW_gate_up", "dW_down", "d_shared_gate_up", "d_shared_down")):
            pairs.append(("layer %d %s" % (i, name), got[i][name], want[1 + i * len(names) + k]))
    for name, a, b in pairs:
        far = ((a.double() - b).norm() / b.norm()).item()
        assert far <= (15 * L) ** 0.5 * 2.0 ** -8, "%s off by %.3g" % (name, far)
