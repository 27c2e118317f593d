"""Keys and queries of very different sizes whose products are ordinary numbers: no intermediate passes fp32's range where the
scores do not, and few and many rows agree."""
import pytest
import torch

import kv4_ref
import ternary_weight_bit_b200 as tb
from kv4_ref import Batch
from test_kv4_gpu import DEV, DTYPES, _clean_status, check_attention, copies, queries, rows_like_keys, rubbish_cache, run_attention  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [1, 30, 200])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("size", [1e-30, 1e-20, 1e20, 1e28, 1e33])
def test_large_keys_and_small_queries(size, dim, dtype, new):
    m = 260
    batch = Batch([m], [m], 64)
    c = rubbish_cache(batch.pages, 2, dim, 64)
    k, v = rows_like_keys((m, 2, dim), 21) * size, rows_like_keys((m, 2, dim), 22)
    tb.bitnet_kv4_write(k.to(DEV), v.to(DEV), c, *batch.tensors(DEV), eps=1e-5 if size > 1 else 1e-36)
    held = copies(c)
    held = [tuple(kv4_ref.values(held[s + "_codes"], held[s + "_step"], held[s + "_bos"], batch, 0) for s in "kv")]
    q = (queries(new, 4, dim, "fp32") * (1 / size)).to(DTYPES[dtype])
    batch = Batch([m], [new], 64)
    out, lse = run_attention(batch, c, q)
    check_attention(batch, c, held, q, out, lse, dim ** -0.5, True, 0)


@pytest.mark.parametrize("new", [1, 30, 200])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_queries_up_to_the_largest_number(dim, dtype, new):
    m = 260
    batch = Batch([m], [m], 64)
    c = rubbish_cache(batch.pages, 2, dim, 64)
    k, v = rows_like_keys((m, 2, dim), 23) * 1e-36, rows_like_keys((m, 2, dim), 24)
    tb.bitnet_kv4_write(k.to(DEV), v.to(DEV), c, *batch.tensors(DEV), eps=1e-38)
    held = copies(c)
    held = [tuple(kv4_ref.values(held[s + "_codes"], held[s + "_step"], held[s + "_bos"], batch, 0) for s in "kv")]
    q = queries(new, 4, dim, "fp32")
    q = q / q.abs().amax(-1, keepdim=True) * 3e36
    q = q.to(DTYPES[dtype])
    q[:, 1::2, 5] = torch.finfo(q.dtype).max
    q[:, 3, 9] = -torch.finfo(q.dtype).max
    batch = Batch([m], [new], 64)
    out, lse = run_attention(batch, c, q)
    check_attention(batch, c, held, q, out, lse, dim ** -0.5, True, 0)


@pytest.mark.parametrize("new,length", [(1, 500), (1, 9000), (30, 500), (200, 260), (200, 9000)])  # whole and in parts
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("bits", [3, 4])
def test_values_near_the_largest_number(bits, dim, dtype, new, length):
    # sums of weights times values stay in range where the values' own sum over all positions does
    batch = Batch([length], [length], 64)
    c = rubbish_cache(batch.pages, 1, dim, 64)
    k, v = rows_like_keys((length, 1, dim), 25), rows_like_keys((length, 1, dim), 26)
    v = v / v.abs().sum() * dim * 3e38
    tb.bitnet_kv4_write(k.to(DEV), v.to(DEV), c, *batch.tensors(DEV), bits=bits)
    held = copies(c)
    held = [tuple(kv4_ref.values(held[s + "_codes"], held[s + "_step"], held[s + "_bos"], batch, 0) for s in "kv")]
    q = queries(new, 4, dim, dtype)
    batch = Batch([length], [new], 64)
    out, lse = run_attention(batch, c, q)
    check_attention(batch, c, held, q, out, lse, dim ** -0.5, True, 0)
