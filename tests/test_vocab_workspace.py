"""A workspace of the vocabulary loss sized for more rows serves fewer (a batch's
last, shorter part), forward and backward."""
import pytest
import torch

from group_limited_routing_gb300 import _lib, build, moe, train


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


@pytest.mark.parametrize("H,V", [(8, 777), (64, 50021), (512, 131072), (2048, 131072), (4096, 30000), (8192, 1 << 20)])
@pytest.mark.parametrize("backward", [0, 1])
def test_size_grows_with_the_rows(lib, H, V, backward):
    size, last = lib.moe_vocab_loss_workspace_bytes, 0
    for T in list(range(0, 400)) + list(range(400, 60000, 41)) + [1 << 18, 1 << 20, 3 << 19, 1 << 21]:
        n = size(T, H, V, backward)
        assert n >= last, (T, n, last)
        last = n


@pytest.mark.gpu
def test_head_of_a_longer_batch():
    """VocabHead for 10700 rows called with one fewer, where a piece of the
    vocabulary holds more columns: the bits of a head of that size."""
    T, H, V = 10699, 64, 50021
    g = torch.Generator().manual_seed(1)
    W = (torch.randn(V, H, generator=g) / 8).bfloat16().cuda()
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    t = torch.randint(0, V, (T,), generator=g).cuda()
    d = torch.full((T,), 1.0 / T, device="cuda")
    out = []
    for rows in (T, T + 1):
        head = train.VocabHead(W, rows)
        loss, lse = head(x, t)
        grad = head.backward(d)
        assert head.status() == 0
        out.append((loss, lse, grad["d_hidden"], grad["dW_vocab"]))
    assert all(torch.equal(a, b) for a, b in zip(*out))
