"""Batches of which one sequence is much longer than the others, where every block could have
a row tile of its own: the long ones are shared by several blocks."""

import numpy as np
import pytest

from tests import kv_util as ku
from tests.test_gpu_kv_attention import Case
from tests.test_gpu_kv_cache import host, i32

pytestmark = pytest.mark.gpu

H, D, G, PAGE = 8, 128, 64, 64


def step(longest, width):
    """A decode step of as many sequences as give two row tiles to an SM, one of `longest` tokens
    and the others of 40, in a table for `width` tokens: the output, whether the call was
    cut, and what it is made of."""
    import torch

    import affine_bit_matmul_gb300 as mxq

    seqs = 2 * torch.cuda.get_device_properties(0).multi_processor_count // H
    ctx = [40] * seqs
    ctx[5] = longest
    c = Case([longest, 40], [1, 1], 4 * H, H, D, G, PAGE, seed=longest)
    table = torch.full((seqs, width // PAGE), -1, dtype=torch.int32, device="cuda")
    used = -(-longest // PAGE)
    table[:, 0] = c.table_d[1, 0]
    table[5, :used] = c.table_d[0, :used]
    q = c.q_d[1].expand(seqs, -1, -1).contiguous()
    q[5] = c.q_d[0]
    ws = torch.full((mxq.kv_attention_workspace_bytes(seqs, seqs, 4 * H, H, D),), 0xAB, dtype=torch.uint8, device="cuda")
    status = i32([-1])
    o = host(mxq.kv_attention(q, c.pages_d, table, i32(ctx), group_size=G, workspace=ws, dev_status=status))
    assert int(status.item()) == 0
    return o, not bool((ws == 0xAB).all()), c


@pytest.mark.parametrize("longest,width,cut", [(1500, 2048, False), (2500, 2560, False), (1500, 4096, True),
                                               (1500, 131072, True)])
def test_one_long_sequence_among_short_ones(longest, width, cut):
    o, was_cut, c = step(longest, width)
    assert was_cut == cut  # a call that is not cut leaves the workspace alone
    ref, _, A, B, E = ku.attention(c.q, c.cache, c.table, c.ctx, c.starts, D ** -0.5)
    tol = ku.tolerance(ref, A, B, E, False)
    assert (np.abs(o[5] - ref[0]) <= tol[0]).all()
    for i in (0, 4, 6, len(o) - 1):
        assert (np.abs(o[i] - ref[1]) <= tol[1]).all()
