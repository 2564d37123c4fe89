"""A training step of a stack of MoE layers: the norms around every block, the
layers, the loss over the vocabulary, and the gradients of all of them.

    step = TrainStack(layers, VocabHead(W_vocab, T), w_pre, w_post, gate)
    loss, lse = step(x, target)                # x [T, H]: the residual stream
    grads = step.backward(d_loss)              # d_loss [T]: 1 / n for the mean over n rows

Layer l of L computes, with n_0 = RMS(x) w_pre[0],
    y_l = layer_l(n_l)
    r_{l+1}, n_{l+1} = block_norm(r_l, y_l, gate[l], w_post[l], w_pre[l + 1])
and the head's loss is that of n_L.  Everything runs in the library's kernels
on the current stream; this module only passes tensors between them.  A backward
reads the tensors of its own forward call (x, target and the weights must still
hold what they held then), so layers and head may be called by others in between
and a layer may stand in several places.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import moe


class VocabHead:
    """The vocabulary's weight [V, H] bf16 and the workspaces of its loss over T rows
    at most: __call__(hidden, target) is vocab_loss, backward(d_loss) the gradient of
    the last call, or of an earlier one whose (hidden, target, lse) it is given."""

    def __init__(self, W_vocab, T: int, ignore_index: int = -100):
        V, H = W_vocab.shape
        self.W_vocab, self.ignore_index = W_vocab, ignore_index
        self.device = W_vocab.device
        self.ws = moe.vocab_loss_workspace(T, H, V, device=self.device)
        self.ws_bwd = None
        self._shape = (T, H, V)
        self._last = None

    def __call__(self, hidden, target):
        loss, lse = moe.vocab_loss(hidden, self.W_vocab, target, ignore_index=self.ignore_index, ws=self.ws)
        self._last = (hidden, target, lse)
        return loss, lse

    def backward(self, d_loss, out: Optional[dict] = None, call=None) -> dict:
        """dict(d_hidden [T, H] bf16, dW_vocab [V, H] bf16)."""
        call = call or self._last
        if call is None:
            raise RuntimeError("backward() needs a forward call first")
        if self.ws_bwd is None:
            self.ws_bwd = moe.vocab_loss_workspace(*self._shape, backward=True, device=self.device)
        hidden, target, lse = call
        return moe.vocab_loss_backward(hidden, self.W_vocab, target, lse, d_loss, ignore_index=self.ignore_index,
                                       ws=self.ws_bwd, out=out)

    def status(self) -> int:
        return self.ws.status() | (self.ws_bwd.status() if self.ws_bwd is not None else 0)


class TrainStack:
    """layers: MoELayer objects of one configuration (aux=True adds the balance
    loss; one object may stand in several places); w_pre [L + 1, H], w_post [L, H]
    and gate [L, H] or [L, groups, H] fp32; alpha the residual scale."""

    def __init__(self, layers, head: VocabHead, w_pre, w_post, gate, alpha: float = 1.0, eps: float = 1e-6):
        self.layers = list(layers)
        if not self.layers:
            raise ValueError("a stack needs a layer")
        self.cfg = self.layers[0].cfg
        self.device = self.layers[0].device
        for layer in self.layers:
            if layer.cfg != self.cfg:
                raise ValueError("layers of one configuration expected, got %r and %r" % (self.cfg, layer.cfg))
        L, H = len(self.layers), self.cfg.H
        for name, t, shape in (("w_pre", w_pre, (L + 1, H)), ("w_post", w_post, (L, H))):
            if tuple(t.shape) != shape:
                raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))
        groups = gate.shape[1] if gate.dim() == 3 else 1
        if tuple(gate.shape) not in ((L, H), (L, groups, H)) or groups < 1 or self.cfg.T % groups:
            raise ValueError("gate must have shape %s or (%d, groups, %d), groups dividing T = %d, got %s" %
                             ((L, H), L, H, self.cfg.T, tuple(gate.shape)))
        self.head = head
        self.w_pre, self.w_post = w_pre, w_post
        self.gate = gate if gate.dim() == 3 else gate[:, None, :]
        self.alpha, self.eps = alpha, eps
        self.ws_route = moe.route_backward_workspace(self.cfg, self.device)
        # the norms behind the layers and the one in front of the first, which has no
        # gate: its plan is that of one group, whose partial sums may be more
        size = moe.block_norm_workspace_bytes
        self.ws_norm = moe.SizedWorkspace(max(size(self.cfg.T, H, groups), size(self.cfg.T, H)),
                                          "moe_block_norm_backward", self.device)
        self._saved = None

    def __call__(self, x, target):
        """(loss [T], lse [T]) of the stack on the residual stream x [T, H] (bf16
        or fp32)."""
        r, n = moe.block_norm(x, w_pre=self.w_pre[0], eps=self.eps)
        saved = []
        for i, layer in enumerate(self.layers):
            call = (n, layer.new_routing())
            y = layer(n, routing=call[1])
            saved.append((r, y, call))
            r, n = moe.block_norm(r, y, self.gate[i], self.w_post[i], self.w_pre[i + 1], alpha=self.alpha,
                                  eps=self.eps)
        loss, lse = self.head(n, target)
        self._saved = (x, saved, (n, target, lse))
        return loss, lse

    def aux_loss(self):
        """The last call's balance losses, one per layer ([1] fp32 each)."""
        if self._saved is None:
            raise RuntimeError("aux_loss() needs a forward call first")
        return [call[1][4] for _, _, call in self._saved[1]]

    def backward(self, d_loss, d_aux_loss=None) -> dict:
        """Gradients of the last call for d_loss [T] fp32 (and d_aux_loss [1] fp32,
        the weight of every layer's balance loss): dict(d_x, dW_vocab, dw_pre
        [L + 1, H], dw_post [L, H], d_gate [L, groups, H], layers: per place in
        the stack what moe.backward gives with d_hidden replaced by the whole one,
        and dW_router)."""
        if self._saved is None:
            raise RuntimeError("backward() needs a forward call first")
        x, saved, head_call = self._saved
        head = self.head.backward(d_loss, call=head_call)
        d_n, d_r = head["d_hidden"], None
        d_y = d_n                          # (nobody else has it; the layers' d_hidden are handed back)
        out = dict(dW_vocab=head["dW_vocab"], dw_pre=torch.empty_like(self.w_pre), dw_post=torch.empty_like(self.w_post),
                   d_gate=torch.empty_like(self.gate), layers=[None] * len(self.layers))
        for i in reversed(range(len(self.layers))):
            r, y, call = saved[i]
            hidden, routing = call
            g = moe.block_norm_backward(r, y, self.gate[i], self.w_post[i], self.w_pre[i + 1], d_r, d_n,
                                        alpha=self.alpha, eps=self.eps, ws=self.ws_norm,
                                        out=dict(dw_pre=out["dw_pre"][i + 1], dw_post=out["dw_post"][i],
                                                 d_gate=out["d_gate"][i], d_y=d_y, d_x=d_r))
            d_r = g["d_x"]
            layer = self.layers[i]
            e = layer.backward(d_y, call=call)
            rb = moe.route_backward(self.cfg, hidden, layer.W_router, routing[0], e["d_topk_w"],
                                    d_aux_loss=d_aux_loss, expert_counts=None if d_aux_loss is None else routing[2],
                                    d_hidden_add=e["d_hidden"], W_split=layer.W_split, ws=self.ws_route,
                                    out=dict(d_hidden=e["d_hidden"]))
            e["dW_router"] = rb["dW_router"]
            out["layers"][i] = e
            d_n = rb["d_hidden"]
        g = moe.block_norm_backward(x, None, None, None, self.w_pre[0], d_r, d_n, eps=self.eps, ws=self.ws_norm,
                                    out=dict(dw_pre=out["dw_pre"][0]))
        out["d_x"] = g["d_x"]
        return out

    def status(self) -> int:
        st = self.head.status() | self.ws_route.status()
        for layer in self.layers:
            st |= layer.status()
        return st
