"""The 8-bit products at sizes where each tile is chosen and every CTA, or pair of
CTAs, takes several tiles, so that accumulators and rings are handed on: dense, with
grouped rows and with grouped sums, in bf16 and in fp32 over several parts of K."""
import ctypes

import pytest
import torch

from group_limited_routing_gb300 import _lib, build, scaled
from test_gpu_scaled import close, operand, rnd

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def tile(gradient, M, N, K, E, dtype, sms):
    """(rows, columns) of the tile, and tiles for each CTA or pair."""
    r, c = ctypes.c_int32(), ctypes.c_int32()
    _lib.check(_lib.load().moe_debug_scaled_tile(gradient, M, N, K, E, int(dtype == F32), sms, ctypes.addressof(r),
                                                 ctypes.addressof(c)), "moe_debug_scaled_tile")
    tiles = -(-M // r.value) * -(-N // c.value) * (E if E and gradient else 1)
    return (r.value, c.value), tiles / (sms // 2 if r.value == 256 else sms)


DENSE = [  # M, N, K, type, tile
    (20000, 1024, 4112, BF, (256, 256)), (20000, 1024, 4112, F32, (256, 256)), (4100, 4096, 1040, BF, (256, 224)),
    (4100, 4096, 8208, F32, (256, 224)), (60000, 72, 512, BF, (128, 128)), (60000, 128, 1024, F32, (128, 128)),
    (60000, 128, 128, BF, (128, 64)), (60000, 128, 128, F32, (128, 64))]
ROWS = [  # rows, N, K, E, type, tile
    (20000, 1024, 4112, 8, BF, (256, 256)), (20000, 1024, 4112, 8, F32, (256, 256)), (20000, 1024, 1040, 8, BF, (256, 224)),
    (20000, 1120, 4112, 8, F32, (256, 224)), (40000, 128, 528, 8, BF, (128, 128)), (40000, 128, 528, 8, F32, (128, 128)),
    (20000, 136, 256, 64, BF, (128, 64)), (20000, 136, 256, 64, F32, (128, 64))]
SUMS = [  # M, N, blocks of 128 rows, E, type, tile
    (1024, 512, 80, 40, BF, (256, 256)), (1024, 512, 720, 40, F32, (256, 256)), (1024, 1024, 320, 16, BF, (256, 224)),
    (1024, 1024, 320, 16, F32, (256, 224)), (1024, 1024, 32, 16, F32, (128, 128)), (128, 128, 1000, 500, BF, (128, 128)),
    (128, 128, 1000, 500, F32, (128, 64)), (4096, 4112, 32, 0, F32, (256, 224)), (20000, 1024, 33, 0, F32, (256, 256))]


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def test_the_cases_cover_every_tile():
    """(on the CPU, for 152 SMs)"""
    every = {(256, 256), (256, 224), (128, 128), (128, 64)}
    for cases, gradient in ((DENSE, 0), (ROWS, 0), (SUMS, 1)):
        seen = set()
        for case in cases:
            M, N, K, E, dtype, want = (*case[:3], 0, *case[3:]) if cases is DENSE else case
            got, each = tile(gradient, M, N, K * 128 if gradient else K, E, dtype, 152)
            assert got == want and each > 1.9, (case, got, each)
            seen.add(got)
        assert seen == every


@pytest.mark.parametrize("kw", [dict(M=0), dict(K=0), dict(K=24), dict(N=12), dict(sms=1), dict(E=-1)])
def test_sizes_without_a_tile(kw):
    a = dict(gradient=0, M=64, N=64, K=128, E=0, dtype=BF, sms=152)
    a.update(kw)
    with pytest.raises(_lib.MoeError):
        tile(**a)


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def counts_of(total, E, seed):
    """Sizes of E groups: some empty, one of a single row, most odd ones."""
    g = torch.Generator().manual_seed(seed)
    share = torch.rand(E, generator=g) ** 2
    share[1::7] = 0
    n = (share / share.sum() * total).long()
    n[2] = 1
    n[0] += total - int(n.sum())
    return n.tolist()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,out,want", DENSE)
def test_dense(M, N, K, out, want):
    assert tile(0, M, N, K, 0, out, sms())[0] == want
    a, A = operand(M, K, 1)
    b, B = operand(N, K, 2, scale=0.02)
    ws = scaled.workspace()
    y = scaled.product(a, b, dtype=out, ws=ws)
    close(y, A, B, K, out)
    again = scaled.product(a, b, dtype=out, ws=ws, out=torch.full_like(y, float("nan")))
    assert torch.equal(y, again) and ws.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("rows,N,K,E,out,want", ROWS)
def test_grouped_rows(rows, N, K, E, out, want):
    assert tile(0, rows, N, K, E, out, sms())[0] == want
    counts = counts_of(rows - 5, E, 3)
    ends = [0]
    for c in counts:
        ends.append(ends[-1] + c)
    offsets = torch.tensor(ends, dtype=torch.int32, device=DEV)
    a, A = operand(rows, K, 1)
    b = scaled.quantize(rnd(E, N, K, seed=2, scale=0.05))
    ws = scaled.workspace()
    y = torch.full((rows, N), 7.0, dtype=out, device=DEV)
    scaled.product(a, b, offsets=offsets, dtype=out, ws=ws, out=y)
    B = b.dequantize()
    for e in range(E):
        if counts[e]:
            close(y[ends[e]:ends[e + 1]], A[ends[e]:ends[e + 1]], B[e].double(), K, out)
    assert bool((y[ends[-1]:] == 7.0).all())                  # rows of no group are left
    again = scaled.product(a, b, offsets=offsets, dtype=out, ws=ws, out=torch.full_like(y, 7.0))
    assert torch.equal(y, again) and ws.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,blocks,E,out,want", SUMS)
def test_sums(M, N, blocks, E, out, want):
    assert tile(1, M, N, blocks * 128, E, out, sms())[0] == want
    if E:
        # (rows whose transposed form has this many blocks)
        rows = (blocks - E) * 128
        counts = counts_of(rows, E, 4)
        ends = [0]
        for c in counts:
            ends.append(ends[-1] + c)
        offsets = torch.tensor(ends, dtype=torch.int32, device=DEV)
    else:
        rows, offsets = blocks * 128 - 5, None
    dy, x = rnd(rows, M, seed=5, scale=1e-3), rnd(rows, N, seed=6)
    dy_t, x_t = [scaled.quantize_columns(t, offsets=offsets) for t in (dy, x)]
    del dy, x
    ws = scaled.workspace()
    dW = scaled.weight_gradient(dy_t, x_t, dtype=out, ws=ws)
    A, B = dy_t.dequantize(), x_t.dequantize()
    if not E:
        close(dW, A.double(), B.double(), rows, out)
    else:
        assert tile(1, M, N, dy_t[0].shape[1], E, out, sms())[0] == want
        starts = dy_t.starts.tolist()
        for e in range(E):
            k0, k1 = 128 * starts[e], 128 * starts[e + 1]
            if k0 == k1:
                assert bool((dW[e] == 0).all())
            else:
                close(dW[e], A[:, k0:k1].double(), B[:, k0:k1].double(), k1 - k0, out)
        if blocks >= 18 * E:
            assert max(b - a for a, b in zip(starts, starts[1:])) > 32          # more than two parts of 2048
    again = scaled.weight_gradient(dy_t, x_t, dtype=out, ws=ws, out=torch.full_like(dW, float("nan")))
    assert torch.equal(dW, again) and ws.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,E,out", [(1024, 4112, 0, BF), (1024, 4112, 0, F32), (1024, 1040, 0, BF), (1024, 4112, 8, BF)])
def test_time_out_on_pairs(N, K, E, out):
    """Both CTAs of a pair wind down, and the next call is right."""
    M = 20000
    assert tile(0, M, N, K, E, out, sms())[0][0] == 256
    a, A = operand(M, K, 1)
    b = scaled.quantize(rnd(*([E] if E else []), N, K, seed=2, scale=0.02))
    offsets = torch.tensor([M * e // E for e in range(E + 1)], dtype=torch.int32, device=DEV) if E else None
    ws = scaled.workspace()
    _lib.check(_lib.load().moe_debug_inject_timeout(1), "inject")
    scaled.product(a, b, offsets=offsets, dtype=out, ws=ws)
    assert ws.status() == _lib.MOE_STATUS_TIMEOUT
    y = scaled.product(a, b, offsets=offsets, dtype=out, ws=ws)
    assert ws.status() == 0
    B = b.dequantize().double()
    for e in range(max(E, 1)):
        part = slice(M * e // E, M * (e + 1) // E) if E else slice(0, M)
        close(y[part], A[part], B[e] if E else B, K, out)
