"""The training step (train.TrainStack) against the same formulas in 64 bits
with autograd, the experts chosen as the step chose them; and a few steps of
gradient descent that lower the loss.

Tolerance: between the loss and a gradient lie, per layer, the bf16 roundings
of n, the intermediate, the expert rows, y, G, U, the weighted intermediate,
dG/dU, the rows' gradients, d_hidden, d_y, d_r and r, and of dz and the head's
d_hidden once: 30 for two layers, each at most 2^-8 of its value and independent
of the others, so sqrt(30) 2^-8 in the 2-norm."""
import pytest
import torch

from group_limited_routing_gb300 import moe, train

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 30 ** 0.5 * 2.0 ** -8


def build(T=96, H=512, I=256, L=2, V=777, stream=torch.bfloat16, groups=3, seed=0, aux=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s, scale=1.0: torch.randn(*s, generator=g) * scale  # noqa: E731
    cfg = moe.MoeConfig(T=T, H=H, I=I, Is=I)
    layers = []
    for _ in range(L):
        layers.append(moe.MoELayer(cfg, rnd(cfg.E, H, scale=0.04).to(DEV), None,
                                   rnd(cfg.E, 2 * I, H, scale=0.04).bfloat16().to(DEV),
                                   rnd(cfg.E, I, H, scale=0.04).bfloat16().to(DEV),
                                   rnd(2 * I, H, scale=0.04).bfloat16().to(DEV),
                                   rnd(I, H, scale=0.04).bfloat16().to(DEV), aux=aux))
    head = train.VocabHead(rnd(V, H, scale=0.04).bfloat16().to(DEV), T)
    step = train.TrainStack(layers, head, (1 + rnd(L + 1, H, scale=0.1)).to(DEV), (1 + rnd(L, H, scale=0.1)).to(DEV),
                            (0.6 + rnd(L, groups, H, scale=0.1)).to(DEV), alpha=0.9)
    x = rnd(T, H).to(stream).to(DEV)
    target = torch.randint(0, V, (T,), generator=g)
    target[::7] = -100
    return step, x, target.to(DEV)


def reference(step, x, target, d_loss, d_aux):
    """The step in 64 bits, with gradients of every leaf."""
    f64 = lambda t: t.detach().double().requires_grad_()  # noqa: E731
    leaves = dict(x=f64(x), w_pre=f64(step.w_pre), w_post=f64(step.w_post), gate=f64(step.gate),
                  W_vocab=f64(step.head.W_vocab))
    per = [dict(W_router=f64(a.W_router), gu=f64(a.W_gate_up), down=f64(a.W_down), sgu=f64(a.shared_gate_up),
                sdown=f64(a.shared_down)) for a in step.layers]
    cfg, eps = step.cfg, step.eps
    rms = lambda t: t / (t.pow(2).mean(1, keepdim=True) + eps).sqrt()  # noqa: E731

    def swiglu(n, gu, down):
        h = n @ gu.t()
        a, b = h[:, :cfg.I], h[:, cfg.I:]
        return (torch.nn.functional.silu(a) * b) @ down

    r = leaves["x"]
    n = rms(r) * leaves["w_pre"][0]
    aux = 0.0
    for i, (layer, w) in enumerate(zip(step.layers, per)):
        idx = layer.routing[0].long()
        s = torch.sigmoid(n @ w["W_router"].t())
        c = s.gather(1, idx)
        weight = c / (c.sum(1, keepdim=True) + cfg.eps) * cfg.rsf
        y = swiglu(n, w["sgu"], w["sdown"])
        for e in range(cfg.E):
            t, j = (idx == e).nonzero(as_tuple=True)
            if t.numel():
                y = y.index_add(0, t, weight[t, j, None] * swiglu(n[t], w["gu"][e], w["down"][e]))
        f = layer.routing[2].double() / (cfg.k * cfg.T)
        aux = aux + cfg.E * (f * (s / s.sum(1, keepdim=True)).mean(0)).sum()
        G = leaves["gate"].shape[1]
        gate = leaves["gate"][i].repeat_interleave(cfg.T // G, 0)
        r = step.alpha * r + gate * (rms(y) * leaves["w_post"][i])
        n = rms(r) * leaves["w_pre"][i + 1]
    z = n @ leaves["W_vocab"].t()
    keep = target >= 0
    loss = torch.where(keep, torch.logsumexp(z, 1) - z.gather(1, target.clamp(min=0)[:, None])[:, 0], 0.0)
    total = (loss * d_loss.double()).sum() + (d_aux.double()[0] * aux if d_aux is not None else 0.0)
    flat = list(leaves.values()) + [t for w in per for t in w.values()]
    grads = torch.autograd.grad(total, flat)
    top = dict(zip(leaves, grads))
    rest = iter(grads[len(leaves):])
    return loss.detach(), top, [dict(zip(w, rest)) for w in per]


def near(got, want, name):
    far = ((got.double() - want).norm() / want.norm()).item()
    assert far <= TOL, "%s off by %.3g" % (name, far)


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("aux", [True, False])
def test_gradients(stream, aux):
    step, x, target = build(stream=stream, seed=3)
    loss, lse = step(x, target)
    n = (target >= 0).sum()
    d_loss = torch.full_like(loss, 1.0) / n
    d_aux = torch.tensor([0.02], device=DEV) if aux else None
    g = step.backward(d_loss, d_aux)
    assert step.status() == 0
    want, top, per = reference(step, x, target, d_loss, d_aux)
    near(loss, want, "loss")
    for name, ref in (("d_x", "x"), ("dW_vocab", "W_vocab"), ("dw_pre", "w_pre"), ("dw_post", "w_post"),
                      ("d_gate", "gate")):
        near(g[name], top[ref], name)
    for i, w in enumerate(per):
        e = g["layers"][i]
        for name, ref in (("dW_router", "W_router"), ("dW_gate_up", "gu"), ("dW_down", "down"),
                          ("d_shared_gate_up", "sgu"), ("d_shared_down", "sdown")):
            near(e[name], w[ref], "layer %d %s" % (i, name))


def test_descent():
    """Plain gradient descent on one batch brings the loss down."""
    step, x, target = build(T=128, L=2, V=500, groups=1, seed=5)
    n = (target >= 0).sum()
    first = None
    for _ in range(12):
        loss, _ = step(x, target)
        mean = (loss.sum() / n).item()
        first = first or mean
        g = step.backward(torch.full_like(loss, 1.0) / n, torch.tensor([0.01], device=DEV))
        step.head.W_vocab.sub_((g["dW_vocab"].float() * 2.0).bfloat16())
        step.w_pre.sub_(g["dw_pre"] * 0.5)
        step.w_post.sub_(g["dw_post"] * 0.5)
        step.gate.sub_(g["d_gate"] * 0.5)
        for layer, e in zip(step.layers, g["layers"]):
            layer.W_router.sub_(e["dW_router"] * 0.5)
            layer.prepare()
            layer.W_gate_up.sub_((e["dW_gate_up"] * 0.5).bfloat16())
            layer.W_down.sub_((e["dW_down"] * 0.5).bfloat16())
    assert step.status() == 0
    assert mean < 0.6 * first, (first, mean)


def test_backward_needs_a_forward():
    step, x, target = build()
    with pytest.raises(RuntimeError):
        step.backward(torch.ones(96, device=DEV))
    with pytest.raises(RuntimeError):
        step.head.backward(torch.ones(96, device=DEV))


def test_captured_step():
    """The whole step, forward and backward, replayed from a CUDA graph on new
    inputs gives the eager step's bits."""
    step, x, target = build(T=64, L=1, V=300, groups=2, seed=9)
    _, x2, target2 = build(T=64, L=1, V=300, groups=2, seed=10)
    d_loss = torch.full((64,), 1.0 / 64, device=DEV)
    d_aux = torch.tensor([0.01], device=DEV)

    def run(a, b):
        loss, _ = step(a, b)
        g = step.backward(d_loss, d_aux)
        e = g["layers"][0]
        return [t.clone() for t in (loss, g["d_x"], g["dW_vocab"], g["dw_pre"], g["dw_post"], g["d_gate"],
                                    e["dW_router"], e["dW_gate_up"], e["dW_down"])]

    wants = [run(x, target), run(x2, target2)]
    sx, st = x.clone(), target.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(sx, st)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(sx, st)
    for (a, b), want in zip(((x2, target2), (x, target)), reversed(wants)):
        sx.copy_(a)
        st.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip(out, want):
            assert torch.equal(got, ref)
    assert step.status() == 0
