"""Block tables that are a part of a wider one: as the C entry points take a table_stride, so does the binding."""
import pytest
import torch

import ternary_weight_bit_b200 as tb
from kv4_ref import Batch
from test_kv4_gpu import DEV, _clean_status, filled, queries  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,new", [([300, 40, 129], [1, 3, 2]), ([200], [1]), ([400, 300], [150, 200])])
def test_a_part_of_a_wider_table(lens, new):
    batch = Batch(lens, new, 64)
    c, _ = filled(batch, 2, 64, 64)
    table, at, starts = batch.tensors(DEV)
    B, width = table.shape
    wide = torch.full((B + 2, width + 9), -5, dtype=torch.int32, device=DEV)
    wide[:B, 3:3 + width] = table
    part = wide[:B, 3:3 + width]
    q = queries(batch.rows, 4, 64, "bf16")
    for a, b in zip(tb.bitnet_kv4_read(c, part, at, starts, batch.rows), tb.bitnet_kv4_read(c, table, at, starts, batch.rows)):
        assert torch.equal(a, b)
    assert torch.equal(tb.bitnet_kv4_attention(q, c, part, at, starts), tb.bitnet_kv4_attention(q, c, table, at, starts))
    k = torch.randn((batch.rows, 2, 64), device=DEV)
    tb.bitnet_kv4_write(k, -k, c, part, at, starts)
    one = tb.bitnet_kv4_read(c, table, at, starts, batch.rows)
    tb.bitnet_kv4_write(k, -k, c, table, at, starts)
    for a, b in zip(one, tb.bitnet_kv4_read(c, table, at, starts, batch.rows)):
        assert torch.equal(a, b)


def test_tables_that_are_refused():
    batch = Batch([300, 40], [1, 3], 64)
    c, _ = filled(batch, 2, 64, 64)
    table, at, starts = batch.tensors(DEV)
    for bad in (table.t().contiguous().t(), table.repeat(1, 2)[:, ::2], table[:1].expand(2, -1)):
        with pytest.raises(ValueError, match="block_table"):
            tb.bitnet_kv4_read(c, bad, at, starts, 4)
    for bad in (table.long(), table[0], table[:1], table.cpu(), [table]):
        with pytest.raises((ValueError, TypeError), match="block_table"):
            tb.bitnet_kv4_read(c, bad, at, starts, 4)
