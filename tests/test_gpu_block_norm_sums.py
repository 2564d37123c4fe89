"""Column sums of block_norm's gradient (d_gate, dw_post, dw_pre) over many rows per
block and many chunks per gate row, against 64 bits.

Tolerance, element by element, in half-steps of 2^-24 of the magnitudes summed:
128 for a term (test_gpu_block_norm's for a gradient element), then one for
each addition of the longest chain, which follows from the launch's plan (plan()
below: the rows are cut into chunks, a block takes one chunk or more):
  dw_pre   the rows of a block, then the blocks' partial sums by 256 slices, 4
           exchanges between lanes and 16 warps;
  d_gate   the rows of a chunk, then a gate row's chunks: up to four gate rows by
           the 256 slices as above, more gate rows one after another;
  dw_post  the same, then the gate rows: up to four one by one, more by the 256
           slices as above."""
import pytest
import torch

from group_limited_routing_gb300 import moe
from test_gpu_block_norm import HALF, U, formulas, inputs

pytestmark = pytest.mark.gpu


def up(a, b):
    return -(-a // b)


def plan(T, H, groups):
    """Blocks and chunks per gate row: the fewest rows in the longest-working block,
    of equal ones the most chunks that give each block one."""
    vectors = H // 8
    threads = up(up(vectors, 1 if vectors <= 32 else 2), 32) * 32
    most, rows, best = 152 * (512 // threads), T // groups, None
    for m in range(5):
        cpg = min(max(m * most // groups if m else 1, 1), rows)
        chunks = groups * cpg
        cost = up(chunks, most) * up(rows, cpg)
        if best is None or cost < best[0] or (cost == best[0] and chunks <= most):
            best = (cost, cpg, min(chunks, most))
    return best


@pytest.mark.parametrize("T,H,groups,stream", [
    (32768, 2048, 1, torch.bfloat16), (32768, 2048, 8, torch.bfloat16), (8192, 1536, 4, torch.float32),
    (65536, 256, 8, torch.bfloat16), (65536, 256, 1, torch.float32), (16384, 256, 64, torch.float32),
    (20000, 512, 5, torch.bfloat16), (20480, 264, 16, torch.bfloat16), (6000, 512, 6000, torch.bfloat16),
    (9000, 4096, 300, torch.bfloat16),
])
def test_column_sums(T, H, groups, stream):
    d = inputs(T, H, groups, stream, seed=T + groups)
    got = moe.block_norm_backward(d["x"], d["y"], d["gate"], d["w_post"], d["w_pre"], d["d_r"], d["d_n"], alpha=0.9)
    longest, cpg, blocks = plan(T, H, groups)
    join = 4 + 16
    chunk = up(T // groups, cpg)
    gate = chunk + (up(cpg, 256) + join if groups <= 4 else cpg)
    steps = dict(d_x=128, d_y=128, dw_pre=128 + longest + up(blocks, 256) + join, d_gate=128 + gate,
                 dw_post=128 + gate + (groups if groups <= 4 else up(groups, 256) + join))
    o, m = formulas(d, 0.9, 1e-6)
    for name, t in got.items():
        bound = HALF[t.dtype] * o[name].abs() + steps[name] * U * m[name] + 1e-37
        over = ((t.double() - o[name]).abs() / bound).max().item()
        assert over <= 1.0, "%s off by %.3g of its bound" % (name, over)
