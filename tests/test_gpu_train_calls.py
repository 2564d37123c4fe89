"""What a training step's backward returns and what it reads of its forward call."""
import pytest
import torch

from group_limited_routing_gb300 import moe, train
from test_gpu_train import DEV, build, near

pytestmark = pytest.mark.gpu


def grads_of_block_inputs(step, x, target, d_loss, d_aux):
    """The step in 64 bits, the experts chosen as the step chose them: the gradient
    of what enters each layer (n_i), by autograd."""
    f64 = lambda t: t.detach().double()  # noqa: E731
    cfg, eps = step.cfg, step.eps
    rms = lambda t: t / (t.pow(2).mean(1, keepdim=True) + eps).sqrt()  # noqa: E731

    def swiglu(n, gu, down):
        a, b = (n @ gu.t()).split(cfg.I, dim=1)
        return (torch.nn.functional.silu(a) * b) @ down

    r = f64(x)
    n = (rms(r) * f64(step.w_pre[0])).requires_grad_()
    ins, aux = [], 0.0
    for i, layer in enumerate(step.layers):
        ins.append(n)
        idx = layer.routing[0].long()
        s = torch.sigmoid(n @ f64(layer.W_router).t())
        c = s.gather(1, idx)
        weight = c / (c.sum(1, keepdim=True) + cfg.eps) * cfg.rsf
        y = swiglu(n, f64(layer.shared_gate_up), f64(layer.shared_down))
        for e in range(cfg.E):
            t, j = (idx == e).nonzero(as_tuple=True)
            if t.numel():
                y = y.index_add(0, t, weight[t, j, None] * swiglu(n[t], f64(layer.W_gate_up[e]), f64(layer.W_down[e])))
        f = layer.routing[2].double() / (cfg.k * cfg.T)
        aux = aux + cfg.E * (f * (s / s.sum(1, keepdim=True)).mean(0)).sum()
        gate = f64(step.gate[i]).repeat_interleave(cfg.T // step.gate.shape[1], 0)
        r = step.alpha * r + gate * (rms(y) * f64(step.w_post[i]))
        n = rms(r) * f64(step.w_pre[i + 1])
    z = n @ f64(step.head.W_vocab).t()
    keep = target >= 0
    loss = torch.where(keep, torch.logsumexp(z, 1) - z.gather(1, target.clamp(min=0)[:, None])[:, 0], 0.0)
    return torch.autograd.grad((loss * d_loss.double()).sum() + d_aux.double()[0] * aux, ins)


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_every_layers_d_hidden(stream):
    """The returned d_hidden of each layer is the gradient of its input through
    experts and router (tolerance: the step's, test_gpu_train)."""
    step, x, target = build(L=3, stream=stream, seed=4)
    loss, _ = step(x, target)
    d_loss = torch.full_like(loss, 1.0) / (target >= 0).sum()
    d_aux = torch.tensor([0.02], device=DEV)
    g = step.backward(d_loss, d_aux)
    assert step.status() == 0
    for i, want in enumerate(grads_of_block_inputs(step, x, target, d_loss, d_aux)):
        near(g["layers"][i]["d_hidden"], want, "layer %d d_hidden" % i)
    tensors = [t for e in g["layers"] for t in e.values()] + [v for k, v in g.items() if k != "layers"]
    assert len({t.data_ptr() for t in tensors}) == len(tensors)      # nothing handed back shares memory


def twin(layer):
    """Another layer object over the same weights."""
    return moe.MoELayer(layer.cfg, layer.W_router, layer.expert_bias, layer.W_gate_up, layer.W_down,
                        layer.shared_gate_up, layer.shared_down, aux=layer.aux, single_call=layer.single_call)


def flat(g):
    return [g[k] for k in ("d_x", "dW_vocab", "dw_pre", "dw_post", "d_gate")] + \
        [e[k] for e in g["layers"] for k in sorted(e)]


def same(a, b):
    return len(a) == len(b) and all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("single_call", [True, False])
def test_one_layer_at_two_places(single_call):
    """A layer object that stands twice gives the bits of two objects over the
    same weights."""
    step, x, target = build(L=3, seed=6)
    a, b = step.layers[:2]
    if not single_call:
        a.single_call = b.single_call = False
        a, b = twin(a), twin(b)
    rest = (step.head, step.w_pre, step.w_post, step.gate)
    one, two = (train.TrainStack(layers, *rest, alpha=0.9) for layers in ([a, b, a], [a, b, twin(a)]))
    d_loss, d_aux = torch.full((96,), 1.0 / 96, device=DEV), torch.tensor([0.02], device=DEV)
    want_loss = two(x, target)
    want_aux = [t.clone() for t in two.aux_loss()]
    want = flat(two.backward(d_loss, d_aux))
    assert same(one(x, target), want_loss)
    assert same(one.aux_loss(), want_aux)
    assert not torch.equal(want_aux[0], want_aux[2])
    assert same(flat(one.backward(d_loss, d_aux)), want)


def test_calls_between_a_forward_and_its_backward():
    """Layers and head called on other data, alone and in another stack, before the
    first stack's backward: its gradients are those of its own call, and so are
    the other stack's."""
    step, x, target = build(L=2, seed=7)
    _, x2, target2 = build(L=2, seed=8)
    d_loss, d_aux = torch.full((96,), 1.0 / 96, device=DEV), torch.tensor([0.02], device=DEV)
    other = train.TrainStack(step.layers, step.head, step.w_pre, step.w_post, step.gate, alpha=0.9)
    losses, wants, auxes = [], [], []
    for a, t in ((x, target), (x2, target2)):
        losses.append(step(a, t))
        auxes.append([v.clone() for v in step.aux_loss()])
        wants.append(flat(step.backward(d_loss, d_aux)))
    step(x, target)
    other(x2, target2)
    n = moe.rmsnorm(x2.bfloat16())
    for layer in step.layers:
        layer(n)
        layer(n.flip(0).contiguous())
    step.head(n, target2)
    assert same(step.aux_loss(), auxes[0]) and same(other.aux_loss(), auxes[1])
    assert same(flat(step.backward(d_loss, d_aux)), wants[0])
    assert same(flat(other.backward(d_loss, d_aux)), wants[1])
    assert same(flat(step.backward(d_loss, d_aux)), wants[0])        # and again


def test_a_captured_layer_keeps_its_routing_tensors():
    """A graph of a layer's call writes the tensors that it was captured with: a
    step in between neither frees them nor has its own overwritten by a replay."""
    step, x, target = build(L=1, seed=9)
    layer = step.layers[0]
    d_loss = torch.full((96,), 1.0 / 96, device=DEV)
    step(x, target)
    want = flat(step.backward(d_loss))
    n = moe.rmsnorm(torch.randn(96, 512, device=DEV).bfloat16())
    eager = layer(n).clone()
    graph = moe.GraphedStep(layer, n)
    mine = layer.routing
    step(x, target)
    assert all(a.data_ptr() != b.data_ptr() for a, b in zip(layer.routing, mine))
    assert torch.equal(graph(n), eager)
    torch.cuda.synchronize()
    assert same(flat(step.backward(d_loss)), want)
    layer(n)
    assert all(a.data_ptr() == b.data_ptr() for a, b in zip(layer.routing, mine))


def test_feedback_after_a_step():
    """layer.routing is the last call's, a step's too: expert_feedback follows it."""
    step, x, target = build(L=1, seed=10)
    layer = step.layers[0]
    layer(moe.rmsnorm(x.flip(0).contiguous()))
    step(x, target)
    totals = torch.zeros(layer.cfg.E, dtype=torch.int64, device=DEV)
    layer.feedback(0.001, totals)
    counts = torch.bincount(step.layers[0].routing[0].flatten().long(), minlength=layer.cfg.E)
    assert torch.equal(totals, counts)


def test_first_norm_of_a_stack_with_several_gates():
    """Three gate rows at a size where the norm without a gate needs more workspace
    than those with; the last step is that norm's gradient, bit for bit."""
    step, x, target = build(T=3000, H=512, I=256, L=1, V=300, groups=3, seed=2, stream=torch.float32)
    step(x, target)
    g = step.backward(torch.full((3000,), 1.0 / 3000, device=DEV))
    assert step.status() == 0
    size = moe._lib.load().moe_block_norm_workspace_bytes
    assert size(3000, 512, 1) > size(3000, 512, 3)
    assert g["d_x"].shape == x.shape and g["d_x"].isfinite().all() and g["dw_pre"].isfinite().all()
