"""The training operators and what surrounds a call: workspaces with other bytes
in them, workspaces of larger calls, workspaces that are too small, outputs with
NaN in them, and calls that follow each other without a pause.  Every result is
the same bits as the first call's with a workspace of its own."""
import pytest
import torch

from group_limited_routing_gb300 import _lib, moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


def loss_case(T, H, V, seed):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(T, H, generator=g).bfloat16().to(DEV)
    W = (torch.randn(V, H, generator=g) / H ** 0.5).bfloat16().to(DEV)
    t = torch.randint(0, V, (T,), generator=g)
    t[torch.rand(T, generator=g) < 0.3] = -100
    t = t.to(DEV)
    d = torch.rand(T, generator=g).to(DEV)

    def run(ws, outs):
        f, b = ws or (None, None)
        loss, lse = moe.vocab_loss(h, W, t, ws=f, out=outs and outs[:2])
        r = moe.vocab_loss_backward(h, W, t, lse, d, ws=b, out=outs and dict(d_hidden=outs[2], dW_vocab=outs[3]))
        return [loss, lse, r["d_hidden"], r["dW_vocab"]]

    return run, lambda: (moe.vocab_loss_workspace(T, H, V), moe.vocab_loss_workspace(T, H, V, backward=True))


def norm_case(T, H, groups, seed):
    g = torch.Generator().manual_seed(seed)
    x, dr = (torch.randn(T, H, generator=g).to(DEV) for _ in range(2))
    y, dn = (torch.randn(T, H, generator=g).bfloat16().to(DEV) for _ in range(2))
    gate, post, pre = (torch.randn(*s, generator=g).to(DEV) for s in ((groups, H), (H,), (H,)))
    names = ("d_x", "d_y", "d_gate", "dw_post", "dw_pre")

    def run(ws, outs):
        r = moe.block_norm_backward(x, y, gate, post, pre, dr, dn, ws=ws and ws[0],
                                    out=outs and dict(zip(names, outs)))
        return [r[n] for n in names]

    return run, lambda: (moe.block_norm_workspace(T, H, groups),)


def route_case(T, H, E, seed):
    g = torch.Generator().manual_seed(seed)
    cfg = moe.MoeConfig(T=T, H=H, E=E, n_group=E // 32, topk_group=max(1, E // 64), k=8)
    h, add = (torch.randn(T, H, generator=g).bfloat16().to(DEV) for _ in range(2))
    W = (torch.randn(E, H, generator=g) / H ** 0.5).to(DEV)
    dw = torch.randn(T, 8, generator=g).to(DEV)
    aux = torch.tensor([0.3], device=DEV)
    idx, _, counts, _, _ = moe.route(cfg, h, W)

    def run(ws, outs):
        r = moe.route_backward(cfg, h, W, idx, dw, d_aux_loss=aux, expert_counts=counts, d_hidden_add=add,
                               ws=ws and ws[0], out=outs and dict(d_hidden=outs[0], dW_router=outs[1]))
        return [r["d_hidden"], r["dW_router"]]

    return run, lambda: (moe.route_backward_workspace(cfg),)


CASES = [(loss_case, (20, 128, 515)), (loss_case, (700, 256, 5000)), (norm_case, (96, 1536, 3)),
         (norm_case, (1000, 512, 100)), (route_case, (16, 256, 256)), (route_case, (100, 320, 256)),
         (route_case, (1500, 256, 128))]


def dirty(ws, byte):
    """Everything but the header, which an owner never writes."""
    ws.buf.fill_(byte)
    _lib.check(_lib.load().moe_workspace_init(ws.ptr, ws.nbytes, torch.cuda.current_stream().cuda_stream), "init")


@pytest.mark.parametrize("case,size", CASES)
@pytest.mark.parametrize("byte", [0, 0x7F, 0xFF])
def test_other_bytes_in_workspace_and_outputs(case, size, byte):
    run, spaces = case(*size, seed=1)
    want = run(None, None)
    ws = spaces()
    for w in ws:
        dirty(w, byte)
    outs = [torch.full_like(t, float("nan")) for t in want]
    got = run(ws, outs)
    assert all(a is b for a, b in zip(got, outs))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(w.status() == 0 for w in ws)


@pytest.mark.parametrize("case,size", CASES)
def test_a_larger_workspace_serves_and_a_smaller_is_refused(case, size):
    run, spaces = case(*size, seed=2)
    want = run(None, None)
    need = [w.nbytes for w in spaces()]
    large = tuple(moe.SizedWorkspace(n + 4096, "test") for n in need)
    for w in large:
        dirty(w, 0xFF)
    assert all(torch.equal(a, b) for a, b in zip(run(large, None), want))
    with pytest.raises(ValueError, match="too small"):
        run(tuple(moe.SizedWorkspace(n - 256, "test") for n in need), None)


@pytest.mark.parametrize("case,sizes", [
    (loss_case, [(700, 256, 5000), (20, 128, 515), (300, 256, 700)]),
    (norm_case, [(96, 1536, 3), (3000, 512, 1), (1000, 512, 100)]),
    (route_case, [(4096, 512, 256), (100, 320, 256), (16, 256, 256), (1500, 256, 128)]),
])
def test_calls_one_after_the_other_in_one_workspace(case, sizes):
    """40 calls of changing sizes, nothing between them: each must find its inputs
    and leave its outputs whole although the next call's kernels overwrite the
    workspace."""
    cases = [case(*s, seed=3 + i) for i, s in enumerate(sizes)]
    want = [run(None, None) for run, _ in cases]
    need = [[w.nbytes for w in spaces()] for _, spaces in cases]
    ws = tuple(moe.SizedWorkspace(max(n), "test") for n in zip(*need))
    torch.cuda.synchronize()
    got = [(i % len(cases), cases[i % len(cases)][0](ws, None)) for i in range(40)]
    torch.cuda.synchronize()
    for i, g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
