"""What a training step's backward returns and what it reads of its forward call."""
import pytest
import torch

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
