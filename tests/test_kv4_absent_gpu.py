"""Rows of the 4-bit cache that are nowhere read as zeros: the number 0, not -0."""
import pytest
import torch

import ternary_weight_bit_b200 as tb
from kv4_ref import Batch
from test_kv4_gpu import DEV, DTYPES, filled
from ternary_weight_bit_b200 import _native

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,rows", [(2, 40), (1, 40000)])  # few heads of many rows have blocks of their own
def test_rows_that_are_nowhere_read_as_zero(heads, rows, dim, dtype):
    batch = Batch([100], [rows], 16)  # the first rows stand before position 0
    c, _ = filled(Batch([100], [1], 16), heads, dim, 16)
    table, lens, starts = batch.tensors(DEV)
    table[0, 5] = -1  # positions 80 .. 95 have no page
    k, v = tb.bitnet_kv4_read(c, table, lens, starts, rows, dtype=DTYPES[dtype])
    assert tb.bitnet_get_last_device_status() == _native.ERR_INVALID_ARG
    pos = torch.arange(100 - rows, 100, device=DEV)
    gone = (pos < 0) | ((pos >= 80) & (pos < 96))
    assert gone.any()
    for y in (k, v):
        y = y[gone]
        assert not y.any() and not torch.signbit(y).any()
