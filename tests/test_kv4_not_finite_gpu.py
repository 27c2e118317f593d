"""Steps and queries of the 4-bit cache's attention that are not finite: the rows that see one are NaN, whatever the signs of
their products (an infinite score of the lower sign must not pass for a hidden position), and no other row changes by a bit.

One new token is the rows kernel's, 30 are so as well, 200 are the tcgen05 kernel's (bf16, dim 64 and 128) or the chunk kernel's."""
import math

import pytest
import torch

import ternary_weight_bit_b200 as tb
from kv4_ref import Batch
from test_kv4_gpu import DEV, DTYPES, _clean_status, filled, queries, rows_like_keys, run_attention  # noqa: F401

pytestmark = pytest.mark.gpu

INF = math.inf


@pytest.mark.parametrize("new", [1, 30, 200])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("pos", [0, 5, 250])
def test_an_infinite_key_step_makes_the_rows_that_see_it_nan(pos, dim, dtype, new):
    batch = Batch([300], [new], 64)
    c, _ = filled(batch, 2, dim, 64)
    q = queries(new, 4, dim, dtype)
    at = torch.arange(300 - new, 300)
    for window in (0, 60):
        want = run_attention(batch, c, q, window=window)
        sees = ((at >= pos) & ((at - pos < window) | (window == 0))).to(DEV)
        for bad in (INF, -INF):  # of the two, one gives a product of the lower sign
            step = c.k_step[int(batch.table[0, pos // 64]), 1]
            kept = step[pos % 64].clone()
            step[pos % 64] = bad
            got = run_attention(batch, c, q, window=window)
            step[pos % 64] = kept
            for g, w in zip(got, want):
                assert g[sees, 2:].isnan().all(), (window, bad)
                assert torch.equal(g[:, :2], w[:, :2]) and torch.equal(g[~sees], w[~sees])


@pytest.mark.parametrize("new", [1, 200])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bits", [3, 4])
def test_a_written_key_with_an_infinite_value_is_not_lost(bits, dtype, new):
    # the write keeps such a key as an infinite step with one code that is not 0: every query sees it, of either sign
    k, v = (rows_like_keys((300, 1, 128), s) for s in (1, 2))
    k[70, 0, 9] = INF
    batch = Batch([300], [300], 64)
    c = tb.KV4Cache.empty(batch.pages, 1, 128)
    tb.bitnet_kv4_write(k.to(DEV), v.to(DEV), c, *batch.tensors(DEV), bits=bits)
    batch = Batch([300], [new], 64)
    q = queries(new, 8, 128, dtype)
    q[:, :4, 9], q[:, 4:, 9] = 1.0, -1.0
    out, lse = run_attention(batch, c, q)
    sees = (torch.arange(300 - new, 300) >= 70).to(DEV)
    assert out[sees].isnan().all() and lse[sees].isnan().all()
    assert out[~sees].isfinite().all() and lse[~sees].isfinite().all()


@pytest.mark.parametrize("new", [1, 30, 200])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_an_infinite_query_makes_its_row_nan(dim, dtype, new):
    # codes of one sign in the dimension where the query is infinite, so that all its scores are so too
    m = 200
    k, v = (rows_like_keys((m, 2, dim), s) for s in (1, 2))
    k[:, 0, 7], k[:, 1, 7] = 4.0, -4.0
    whole = Batch([m], [m], 32)
    c = tb.KV4Cache.empty(whole.pages, 2, dim, page_size=32)
    tb.bitnet_kv4_write(k.to(DEV), v.to(DEV), c, *whole.tensors(DEV))
    batch = Batch([m], [new], 32)
    good = queries(new, 4, dim, dtype)
    for window in (0, 1, 50):
        for causal in (True, False) if window == 0 else (True,):
            want = run_attention(batch, c, good, causal=causal, window=window)
            for bad in (INF, -INF, math.nan):
                q = good.clone()
                rows = sorted({0, new // 2, new - 1})
                q[rows, 1, 7], q[rows, 2, 7] = bad, bad
                got = run_attention(batch, c, q, causal=causal, window=window)
                keep = torch.ones(q.shape[:2], dtype=torch.bool, device=DEV)
                keep[rows, 1:3] = False
                for g, w in zip(got, want):
                    assert g[rows, 1:3].isnan().all(), (window, causal, bad)
                    assert torch.equal(g[keep], w[keep])


@pytest.mark.parametrize("new", [3, 200])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_row_that_sees_nothing_is_zero_whatever_its_query(dim, dtype, new):
    batch = Batch([new - 2], [new], 32)  # the first two rows stand before the cache
    c, _ = filled(batch, 2, dim, 32)
    q = queries(new, 4, dim, dtype)
    q[0, :, 3], q[1, :, 5] = INF, math.nan
    out, lse = run_attention(batch, c, q)
    assert not out[:2].any() and (lse[:2] == -INF).all()
    assert out[2:].isfinite().all() and lse[2:].isfinite().all()
