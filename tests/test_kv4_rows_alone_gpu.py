"""A row of the 4-bit cache's attention does not depend on the other rows of its call: whatever their queries are, it has the
same bits.  (Rows that share a key head share tiles, loops and a vote on moving their references.)"""
import math

import pytest
import torch

from kv4_ref import Batch
from test_kv4_gpu import DEV, _clean_status, filled, queries, run_attention  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [1, 3, 30, 200])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_row_has_the_same_bits_beside_any_others(dim, dtype, new):
    batch = Batch([570], [new], 64)  # short enough that an item is one CTA's, whose warps walk several tiles each
    c, _ = filled(batch, 1, dim, 64)
    q = queries(new, 8, dim, dtype) * 4  # scores that pass the references now and then
    mine = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    mine[::2, 1::3] = True
    want = run_attention(batch, c, q)
    for factor in (0.0, 1e-3, -30.0, math.nan):
        other = torch.where(mine[..., None], q, q * factor)
        for g, w in zip(run_attention(batch, c, other), want):
            assert torch.equal(g[mine], w[mine]), factor
