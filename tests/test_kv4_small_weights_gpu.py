"""Weights far below their row's largest in bf16 calls: how finely the 4-bit cache's attention holds them.

A weight times its value's step is held in fp16, over a power of two 2^e.  The row's largest weight stands at 2^6 at least, so what
falls below fp16's normal numbers is off by at most 2^-25 of 2^-6: 2^-31 of the row's largest weight, times 2^e."""
import pytest
import torch

import kv4_ref
import ternary_weight_bit_b200 as tb
from kv4_ref import Batch
from test_kv4_gpu import DEV, _clean_status, copies, rubbish_cache, run_attention  # noqa: F401

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def cache_of(k, v, page):
    m, heads, dim = k.shape
    batch = Batch([m], [m], page)
    c = rubbish_cache(batch.pages, heads, dim, page)
    tb.bitnet_kv4_write(k.to(DEV), v.to(DEV), c, *batch.tensors(DEV))
    held = copies(c)
    return c, [kv4_ref.values(held[s + "_codes"], held[s + "_step"], held[s + "_bos"], batch, 0) for s in "kv"], held


def reference(q, k, v):
    """(out, bound without the smallest weights' term) of queries at the last positions."""
    out, _, top, mass = kv4_ref.attention(q.cpu().float(), k, v, k.shape[-1] ** -0.5, True, 0)
    err, _ = kv4_ref.attention_bounds(out, top, mass, k.shape[-1], k.shape[0], BF16, 0.0)
    return out, err


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 8, 200])
def test_weights_far_below_the_largest(new, dim):
    # one position of the largest weight and a value of zero; all others 2^-18 to 2^-27 of it, with values of one sign
    m, heads = 900, 16
    sign = torch.where(torch.randn(dim, generator=torch.Generator().manual_seed(1)) > 0, 1.0, -1.0)
    k, v = -sign.expand(m, 1, dim).clone(), torch.ones((m, 1, dim))
    k[3], v[3] = sign, 0.0
    c, (kv, vv), _ = cache_of(k, v, 64)
    gap = float((kv[3, 0] - kv[5, 0]) @ sign.double()) * dim ** -0.5  # of scores, for a query `sign`
    size = torch.linspace(18.0, 27.0, heads) * 0.6931471805599453 / gap
    q = (size[None, :, None] * sign).expand(new, heads, dim).to(BF16).to(DEV)
    got, _ = run_attention(Batch([m], [new], 64), c, q)
    want, err = reference(q, kv, vv)
    err = err + 2.0 ** -31 * vv.abs().sum(0)[None]  # every step but that of the zero row is one and the same
    off = (got.cpu().double() - want).abs()
    assert (off <= err).all(), float((off / err).max())
