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


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 8])
@pytest.mark.parametrize("m,size", [(500, 28), (570, 29), (3000, 28)])
def test_a_large_value_step_touches_its_own_tile_alone(m, size, new, dim):
    # Values 2^28 times the others' at positions whose weight is 0, one in each warp's first tile of 32 positions: few rows hold
    # what follows them as finely as without them.  2^e is the power of two of the largest step of a tile.
    g = torch.Generator().manual_seed(2)
    sign = torch.where(torch.randn(dim, generator=g) > 0, 1.0, -1.0)
    k, v = sign.expand(m, 1, dim).clone(), 1.0 + torch.rand((m, 1, dim), generator=g)
    for pos in (5, 40, 70, 100):
        k[pos], v[pos] = -sign, v[pos] * 2.0 ** size
    c, (kv, vv), held = cache_of(k, v, 32)
    gap = float((kv[7, 0] - kv[5, 0]) @ sign.double()) * dim ** -0.5
    q = (sign * (60 * 0.6931471805599453 / gap)).expand(new, 8, dim).to(BF16).to(DEV)  # 2^-60 for the large
    batch = Batch([m], [new], 32)
    got, _ = run_attention(batch, c, q)
    want, err = reference(q, kv, vv)
    at, off = Batch([m], [m], 32).table[0].long()[torch.arange(m) // 32], torch.arange(m) % 32
    step = held["v_step"][at, 0, off].double()
    code = vv.abs()[:, 0] / step[:, None]
    large = torch.cat([s.max().log2().floor().exp2().expand(s.numel()) for s in step.split(32)])
    # m - 5 positions of the largest weight (position 0, at 8 bits, has less), so each is off by 2^-31 2^e |code| over their number
    err = err + (2.0 ** -31 * large[:, None] * code).sum(0) / (m - 5)
    d = (got.cpu().double() - want).abs()
    assert (d <= err).all(), float((d / err).max())
