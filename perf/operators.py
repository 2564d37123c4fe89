"""What is measured of the training operators beside the MoE layer: the
vocabulary loss and its gradient, the norms around a block with its gate and
residual scale and their gradient, and the router's gradient.

Each case runs one operator once, on inputs drawn from a seed.  With `own`
false, run() computes it with elementary torch operations in 32 bits; with
`own` true it makes the calls a user makes of group_limited_routing_gb300.moe.
"""
import math

import torch

own = False

DEV = "cuda"
IGNORE = -100


# ------------------------------------------------------------------- cases
def listed():
    return [
        # ---- loss of the last hidden states over the vocabulary
        # a test-sized model's step: latency
        dict(name="loss_tiny", op="loss", T=128, H=512, V=1000, ignored=0.0),
        # a few rows scored against a full vocabulary: streams the head's weight
        dict(name="loss_few_rows", op="loss", T=16, H=2048, V=131072, ignored=0.0),
        # a training batch
        dict(name="loss_batch", op="loss", T=8192, H=2048, V=131072, ignored=0.05),
        # its gradient, on a ragged batch whose prompt rows carry no loss
        dict(name="loss_bwd_ragged", op="loss_bwd", T=1021, H=1536, V=50021, ignored=0.4),
        # its gradient on a training batch
        dict(name="loss_bwd_batch", op="loss_bwd", T=8192, H=2048, V=65536, ignored=0.05),
        # ---- norms around a block
        # a decode-sized step of the full-size layer
        dict(name="norm_decode", op="norm", T=16, H=2048, gates=1, stream="bf16"),
        # the full-size layer's batch
        dict(name="norm_batch", op="norm", T=32768, H=2048, gates=1, stream="bf16"),
        # gradient, ragged, one gate vector for each of 3 sequences, fp32 stream
        dict(name="norm_bwd_ragged", op="norm_bwd", T=4095, H=1536, gates=3, stream="fp32"),
        # gradient on the full-size layer's batch
        dict(name="norm_bwd_batch", op="norm_bwd", T=32768, H=2048, gates=1, stream="bf16"),
        # ---- the router's gradient
        # the tiny layer
        dict(name="route_bwd_tiny", op="route_bwd", T=128, H=512, E=256, k=8, aux=True, add=True),
        # two packed sequences, no balance loss
        dict(name="route_bwd_seqs", op="route_bwd", T=4096, H=2048, E=256, k=8, aux=False, add=True),
        # the full-size layer's batch, balance loss, added to the experts' gradient
        dict(name="route_bwd_batch", op="route_bwd", T=32768, H=2048, E=256, k=8, aux=True, add=True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["loss", "loss_bwd", "norm", "norm_bwd", "route_bwd"])
    if op in ("loss", "loss_bwd"):
        most = 8192 * 2048 * (131072 if op == "loss" else 65536)
        while True:
            c = dict(op=op, T=_log_int(rng, 1, 16384), H=_log_int(rng, 256, 4096, 8), V=_log_int(rng, 500, 131072),
                     ignored=rng.choice([0.0, 0.0, 0.1, 0.5, 0.9]))
            if c["T"] * c["H"] * c["V"] <= most and c["T"] * c["V"] <= 1 << 30:
                return c
    if op in ("norm", "norm_bwd"):
        while True:
            T = _log_int(rng, 1, 65536)
            c = dict(op=op, T=T, H=_log_int(rng, 256, 8192, 8),
                     gates=rng.choice([1, 1, rng.choice([d for d in range(1, min(T, 64) + 1) if T % d == 0])]),
                     stream=rng.choice(["bf16", "bf16", "fp32"]))
            if c["T"] * c["H"] * (2 if c["stream"] == "fp32" else 1) <= 32768 * 2048:
                return c
    while True:
        c = dict(op=op, T=_log_int(rng, 1, 32768), H=_log_int(rng, 512, 4096, 64), E=rng.choice([128, 256, 256]),
                 k=rng.randint(1, 8), aux=rng.random() < 0.5, add=rng.random() < 0.5)
        if c["T"] * c["H"] <= 32768 * 2048:
            return c


# ------------------------------------------------------------------ inputs
def _bf(t):
    return t.to(torch.bfloat16)


def _prepare_loss(case, g):
    T, H, V = case["T"], case["H"], case["V"]
    W = _bf(torch.randn(V, H, device=DEV, generator=g) * 0.02)
    target = torch.randint(0, V, (T,), device=DEV, generator=g)
    # normalised states that lean towards their target by various amounts, so
    # that the losses run from near zero to above log V
    lean = torch.rand(T, 1, device=DEV, generator=g) * 16.0 / (0.0004 * H)
    hidden = _bf(torch.randn(T, H, device=DEV, generator=g) + lean * W[target].float())
    masked = torch.rand(T, device=DEV, generator=g) < case["ignored"]
    target = torch.where(masked, torch.full_like(target, IGNORE), target)
    s = dict(case=case, hidden=hidden, W=W, target=target)
    if case["op"] == "loss_bwd":
        lse = torch.logsumexp(hidden.float() @ W.float().t(), 1)
        s["lse"] = torch.where(masked, torch.zeros_like(lse), lse)
        # the mean over the rows that count, each with a weight of its own
        n = (~masked).sum().clamp(min=1)
        weight = torch.rand(T, device=DEV, generator=g) * 0.5 + 0.75
        s["d_loss"] = weight / n
    return s


def _prepare_norm(case, g):
    T, H, G = case["T"], case["H"], case["gates"]
    stream = torch.float32 if case["stream"] == "fp32" else torch.bfloat16
    rnd = lambda *shape: torch.randn(*shape, device=DEV, generator=g)  # noqa: E731
    s = dict(case=case, x=(rnd(T, H) * 2.0).to(stream), y=_bf(rnd(T, H) * 0.3), gate=rnd(G, H) * 0.2 + 0.5,
             w_post=rnd(H) * 0.1 + 1.0, w_pre=rnd(H) * 0.1 + 1.0, alpha=0.9, eps=1e-6)
    if case["op"] == "norm_bwd":
        s["d_r"] = (rnd(T, H) * 1e-3).to(stream)
        s["d_n"] = _bf(rnd(T, H) * 1e-3)
    return s


def _prepare_route(case, g):
    T, H, E, k = case["T"], case["H"], case["E"], case["k"]
    n_group, rsf, eps = E // 32, 2.5, 1e-20
    keep = max(1, n_group // 2)
    hidden = _bf(torch.randn(T, H, device=DEV, generator=g))
    W = torch.randn(E, H, device=DEV, generator=g) * 0.02
    score = torch.sigmoid(hidden.float() @ W.t())
    best = score.view(T, n_group, 32).topk(2, dim=2).values.sum(2).topk(keep, dim=1).indices
    alive = torch.zeros(T, n_group, dtype=torch.bool, device=DEV).scatter_(1, best, True)
    alive = alive.repeat_interleave(32, dim=1)
    idx = score.masked_fill(~alive, -1.0).topk(k, dim=1).indices.to(torch.int32)
    counts = torch.bincount(idx.flatten().long(), minlength=E).to(torch.int32)
    s = dict(case=case, hidden=hidden, W=W, idx=idx, counts=counts, rsf=rsf, eps=eps, n_group=n_group, keep=keep,
             d_w=torch.randn(T, k, device=DEV, generator=g) * 1e-3, d_aux=None, add=None)
    if case["aux"]:
        s["d_aux"] = torch.rand(1, device=DEV, generator=g) * 0.01 + 0.005
    if case["add"]:
        s["add"] = _bf(torch.randn(T, H, device=DEV, generator=g) * 1e-3)
    return s


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    if case["op"] in ("loss", "loss_bwd"):
        return _prepare_loss(case, g)
    if case["op"] in ("norm", "norm_bwd"):
        return _prepare_norm(case, g)
    return _prepare_route(case, g)


# ------------------------------------------------------------- plain forms
def _plain_loss(s):
    z = s["hidden"].float() @ s["W"].float().t()
    keep = s["target"] != IGNORE
    lse = torch.logsumexp(z, 1)
    at = z.gather(1, s["target"].clamp(min=0)[:, None])[:, 0]
    return dict(loss=torch.where(keep, lse - at, 0.0), lse=torch.where(keep, lse, 0.0))


def _plain_loss_bwd(s):
    h, W = s["hidden"].float(), s["W"].float()
    keep = s["target"] != IGNORE
    dz = torch.exp(h @ W.t() - s["lse"][:, None])
    dz.scatter_add_(1, s["target"].clamp(min=0)[:, None], torch.full_like(s["lse"], -1.0)[:, None])
    dz *= torch.where(keep, s["d_loss"], 0.0)[:, None]
    return dict(d_hidden=_bf(dz @ W), dW_vocab=_bf(dz.t() @ h))


def _norm_parts(s):
    x, y = s["x"].float(), s["y"].float()
    T, G = x.shape[0], s["gate"].shape[0]
    gate = s["gate"].repeat_interleave(T // G, dim=0)
    rho = torch.rsqrt(y.square().mean(1, keepdim=True) + s["eps"])
    u = y * rho
    v = u * s["w_post"]
    r = s["alpha"] * x + gate * v
    sigma = torch.rsqrt(r.square().mean(1, keepdim=True) + s["eps"])
    return gate, rho, u, v, r, sigma


def _plain_norm(s):
    _, _, _, _, r, sigma = _norm_parts(s)
    return dict(r=r.to(s["x"].dtype), n=_bf(r * sigma * s["w_pre"]))


def _plain_norm_bwd(s):
    gate, rho, u, v, r, sigma = _norm_parts(s)
    G, H = s["gate"].shape
    dn = s["d_n"].float()
    q = r * sigma
    dq = dn * s["w_pre"]
    dr = s["d_r"].float() + sigma * (dq - q * (dq * q).mean(1, keepdim=True))
    dv = dr * gate
    du = dv * s["w_post"]
    return dict(d_x=(s["alpha"] * dr).to(s["x"].dtype), d_y=_bf(rho * (du - u * (du * u).mean(1, keepdim=True))),
                d_gate=(dr * v).view(G, -1, H).sum(1), dw_post=(dv * u).sum(0), dw_pre=(dn * q).sum(0))


def _plain_route_bwd(s):
    x, W, idx = s["hidden"].float(), s["W"], s["idx"].long()
    T, E = x.shape[0], W.shape[0]
    score = torch.sigmoid(x @ W.t())
    chosen = score.gather(1, idx)
    den = chosen.sum(1, keepdim=True) + s["eps"]
    dc = s["rsf"] / den * (s["d_w"] - (s["d_w"] * chosen).sum(1, keepdim=True) / den)
    ds = torch.zeros_like(score).scatter_add_(1, idx, dc)
    if s["d_aux"] is not None:
        f = s["counts"].float() / idx.numel()
        z = score.sum(1, keepdim=True)
        ds = ds + s["d_aux"] * E / T * (f - (score * f).sum(1, keepdim=True) / z) / z
    dl = ds * score * (1 - score)
    dx = dl @ W
    return dict(d_hidden=_bf(dx if s["add"] is None else dx + s["add"].float()), dW_router=dl.t() @ x)


_PLAIN = dict(loss=_plain_loss, loss_bwd=_plain_loss_bwd, norm=_plain_norm, norm_bwd=_plain_norm_bwd,
              route_bwd=_plain_route_bwd)


# --------------------------------------------------------- the framework's
def _own_loss(s, moe):
    if "ws" not in s:
        s["ws"] = moe.vocab_loss_workspace(s["case"]["T"], s["case"]["H"], s["case"]["V"])
    loss, lse = moe.vocab_loss(s["hidden"], s["W"], s["target"], ignore_index=IGNORE, ws=s["ws"])
    return dict(loss=loss, lse=lse)


def _own_loss_bwd(s, moe):
    if "ws" not in s:
        s["ws"] = moe.vocab_loss_workspace(s["case"]["T"], s["case"]["H"], s["case"]["V"], backward=True)
    return moe.vocab_loss_backward(s["hidden"], s["W"], s["target"], s["lse"], s["d_loss"], ignore_index=IGNORE,
                                   ws=s["ws"])


def _own_norm(s, moe):
    r, n = moe.block_norm(s["x"], s["y"], s["gate"], s["w_post"], s["w_pre"], alpha=s["alpha"], eps=s["eps"])
    return dict(r=r, n=n)


def _own_norm_bwd(s, moe):
    if "ws" not in s:
        s["ws"] = moe.block_norm_workspace(s["case"]["T"], s["case"]["H"], s["case"]["gates"])
    return moe.block_norm_backward(s["x"], s["y"], s["gate"], s["w_post"], s["w_pre"], s["d_r"], s["d_n"],
                                   alpha=s["alpha"], eps=s["eps"], ws=s["ws"])


def _own_route_bwd(s, moe):
    c = s["case"]
    if "ws" not in s:
        s["cfg"] = moe.MoeConfig(T=c["T"], H=c["H"], E=c["E"], n_group=s["n_group"], topk_group=s["keep"], k=c["k"],
                                 rsf=s["rsf"], eps=s["eps"])
        s["ws"] = moe.route_backward_workspace(s["cfg"])
    return moe.route_backward(s["cfg"], s["hidden"], s["W"], s["idx"], s["d_w"], d_aux_loss=s["d_aux"],
                              expert_counts=s["counts"], d_hidden_add=s["add"], ws=s["ws"])


_OWN = dict(loss=_own_loss, loss_bwd=_own_loss_bwd, norm=_own_norm, norm_bwd=_own_norm_bwd, route_bwd=_own_route_bwd)


def run(state):
    op = state["case"]["op"]
    if own:
        from group_limited_routing_gb300 import moe
        return _OWN[op](state, moe)
    return _PLAIN[op](state)


# -------------------------------------------------------------------- work
def work(case):
    T, H, op = case["T"], case["H"], case["op"]
    if op in ("loss", "loss_bwd"):
        V = case["V"]
        rows = T * (1.0 - case["ignored"])
        if op == "loss":
            return dict(bytes=2.0 * (rows + V) * H + 16.0 * T, flops=2.0 * rows * V * H)
        return dict(bytes=4.0 * (rows + V) * H + 16.0 * T, flops=6.0 * rows * V * H)
    if op in ("norm", "norm_bwd"):
        el = 4 if case["stream"] == "fp32" else 2
        G = case["gates"]
        if op == "norm":
            return dict(bytes=T * H * (2.0 * el + 4) + 4.0 * H * (G + 2), flops=12.0 * T * H)
        return dict(bytes=T * H * (3.0 * el + 6) + 8.0 * H * (G + 2), flops=36.0 * T * H)
    E, k = case["E"], case["k"]
    return dict(bytes=T * H * (4.0 + (2 if case["add"] else 0)) + 8.0 * E * H + 8.0 * T * k, flops=6.0 * T * E * H)


# -------------------------------------------------- the definitions, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    T, H, op = case["T"], case["H"], case["op"]
    if op in ("loss", "loss_bwd"):
        if (2.0 if op == "loss" else 6.0) * T * H * case["V"] > 7e12:
            return None
        h, W, target = s["hidden"].double(), s["W"].double(), s["target"]
        counted = (target >= 0).nonzero()[:, 0]
        at = target[counted]
        if op == "loss":
            out = dict(loss=torch.zeros(T, dtype=torch.float64, device=DEV),
                       lse=torch.zeros(T, dtype=torch.float64, device=DEV))
            for i in range(0, counted.numel(), 1024):
                rows = counted[i:i + 1024]
                z = h[rows] @ W.t()
                top = z.amax(1)
                lse = top + (z - top[:, None]).exp().sum(1).log()
                out["lse"][rows] = lse
                out["loss"][rows] = lse - (h[rows] * W[target[rows]]).sum(1)
            return out
        d_hidden = torch.zeros(T, H, dtype=torch.float64, device=DEV)
        dW = torch.zeros_like(W)
        weight = s["d_loss"].double()
        for i in range(0, counted.numel(), 1024):
            rows = counted[i:i + 1024]
            p = (h[rows] @ W.t() - s["lse"].double()[rows, None]).exp()
            p[torch.arange(rows.numel(), device=DEV), at[i:i + 1024]] -= 1.0
            p *= weight[rows, None]
            d_hidden[rows] = p @ W
            dW += p.t() @ h[rows]
        return dict(d_hidden=d_hidden, dW_vocab=dW)
    if op in ("norm", "norm_bwd"):
        x, y, eps, alpha = s["x"].double(), s["y"].double(), s["eps"], s["alpha"]
        G = s["gate"].shape[0]
        leaves = [x, y, s["gate"].double(), s["w_post"].double(), s["w_pre"].double()]
        if op == "norm_bwd":
            leaves = [t.requires_grad_() for t in leaves]
        x, y, gate, w_post, w_pre = leaves
        post = y / (y.pow(2).sum(1, keepdim=True) / H + eps).sqrt() * w_post
        r = alpha * x + (gate[:, None, :] * post.view(G, T // G, H)).reshape(T, H)
        n = r / (r.pow(2).sum(1, keepdim=True) / H + eps).sqrt() * w_pre
        if op == "norm":
            return dict(r=r, n=n)
        grads = torch.autograd.grad([r, n], leaves, [s["d_r"].double(), s["d_n"].double()])
        return dict(zip(("d_x", "d_y", "d_gate", "dw_post", "dw_pre"), grads))
    if 6.0 * T * case["E"] * H > 7e12:
        return None
    x, W = s["hidden"].double().requires_grad_(), s["W"].double().requires_grad_()
    score = 1.0 / (1.0 + (-(x @ W.t())).exp())
    chosen = score.gather(1, s["idx"].long())
    total = (chosen / (chosen.sum(1, keepdim=True) + s["eps"]) * s["rsf"] * s["d_w"].double()).sum()
    if s["d_aux"] is not None:
        share = (score / score.sum(1, keepdim=True)).mean(0)
        total = total + s["d_aux"].double()[0] * case["E"] * (s["counts"].double() / (T * case["k"]) * share).sum()
    dx, dW = torch.autograd.grad(total, [x, W])
    return dict(d_hidden=dx if s["add"] is None else dx + s["add"].double(), dW_router=dW)
