"""Many rows behind long contexts: the rings of the tcgen05 kernel (places 8 deep, steps 4, keys and values 2) and of the chunk
kernel turn many times, items are whole or cut into parts of many steps, and references and the units of the outputs
move late.  Against plain 64-bit arithmetic, for some of the heads."""
import math

import pytest
import torch

import kv4_ref
import ternary_weight_bit_b200 as tb
from kv4_ref import U, Batch
from test_kv4_gpu import DEV, _clean_status, check_attention, copies, queries, rows_like_keys, rubbish_cache, run_attention  # noqa: F401

pytestmark = pytest.mark.gpu

FORMS = [("bf16", 64), ("bf16", 128), ("bf16", 256), ("fp32", 64), ("fp32", 128), ("fp32", 256)]


def written(batch, heads, dim, page, k, v, bits=4):
    """A cache that holds rows k, v [positions of all sequences, heads, dim]."""
    c = rubbish_cache(batch.pages, heads, dim, page)
    whole = Batch.__new__(Batch)
    whole.__dict__ = dict(batch.__dict__, new=batch.lens)
    whole.starts = torch.tensor([sum(batch.lens[:i]) for i in range(len(batch.lens) + 1)], dtype=torch.int32)
    tb.bitnet_kv4_write(k.to(DEV), v.to(DEV), c, *whole.tensors(DEV), bits=bits)
    return c


def check_heads(batch, c, q, out, lse, pick, causal=True, window=0):
    """check_attention for the key heads `pick` and their query heads."""
    group = q.shape[1] // c.heads
    held = copies(c)
    values = [tuple(kv4_ref.values(held[s + "_codes"][:, pick], held[s + "_step"][:, pick], held[s + "_bos"][:, pick], batch, b)
                    for s in "kv") for b in range(len(batch.lens))]
    mine = torch.tensor([h * group + i for h in pick for i in range(group)])
    check_attention(batch, c, values, q.cpu()[:, mine], out.cpu()[:, mine], lse.cpu()[:, mine], c.dim ** -0.5, causal, window)


@pytest.mark.parametrize("dtype,dim", FORMS)
@pytest.mark.parametrize("window", [0, 1500])
def test_items_of_many_steps(window, dtype, dim):
    # 286 items of 256 rows or 442 of 128 at most, of which 222 are enough that none is cut: a CTA walks up to 20 steps of 128
    # positions, or 40 of 64
    lens, new = [2500, 2304, 2111, 1900, 2433, 2049], [130, 257, 300, 128, 200, 511]
    batch = Batch(lens, new, 64, lead=3, tail=5)
    heads = 26
    k, v = (rows_like_keys((sum(lens), heads, dim), s) for s in (1, 2))
    c = written(batch, heads, dim, 64, k, v)
    q = queries(batch.rows, heads, dim, dtype)
    out, lse = run_attention(batch, c, q, window=window)
    check_heads(batch, c, q, out, lse, [0, 25], window=window)


@pytest.mark.parametrize("dtype,dim", FORMS)
@pytest.mark.parametrize("page,causal,window", [(16, True, 0), (256, True, 0), (64, True, 5000), (64, False, 0)])
def test_items_cut_into_parts_of_many_steps(page, causal, window, dtype, dim):
    batch = Batch([9001, 4097], [141, 260], page, tail=4)
    k, v = (rows_like_keys((13098, 2, dim), s) for s in (3, 4))
    c = written(batch, 2, dim, page, k, v, bits=3)
    q = queries(batch.rows, 6, dim, dtype)
    out, lse = run_attention(batch, c, q, causal=causal, window=window)
    check_heads(batch, c, q, out, lse, [0, 1], causal, window)


@pytest.mark.parametrize("dtype,dim", FORMS)
@pytest.mark.parametrize("heads", [1, 60])  # cut, and whole
def test_references_and_units_that_move_late(heads, dtype, dim):
    # keys and values that grow by a factor of 2^20 along the sequence, in steps at odd places
    batch = Batch([3000, 2900], [256, 300], 32)
    grow = torch.exp2(torch.cat([torch.arange(m) // 313 * 2.3 for m in batch.lens]))[:, None, None]
    k, v = (rows_like_keys((5900, heads, dim), s) for s in (5, 6))
    c = written(batch, heads, dim, 32, k * grow.sqrt() / 64, v * grow)
    q = queries(batch.rows, heads, dim, dtype)
    out, lse = run_attention(batch, c, q)
    check_heads(batch, c, q, out, lse, [heads - 1])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,m", [(56, 12000), (1, 30000)])  # whole, and cut into eight parts
def test_fp32_sums_of_one_sign_are_not_cut(heads, m, dim):
    """Values of one sign and nearly equal weights: roundings to nearest of such a sum's m terms lie on both sides and add
    up to a few sqrt(m) / 2 of them, roundings that always cut add up to m.  Allowed: what check_attention allows without its
    term for scores, which queries of 1e-3 leave at most 0.1 * 2^-24 each, so 2 sqrt(m) + 32 roundings (251 for 12,000); and
    for the mean over all outputs, whose roundings to nearest have no common sign, one in eight of that."""
    g = torch.Generator(DEV).manual_seed(dim)
    batch = Batch([m], [m], 64)
    k = torch.randn((m, heads, dim), generator=g, device=DEV)
    v = torch.rand((m, heads, dim), generator=g, device=DEV) + 0.5
    c = written(batch, heads, dim, 64, k, v)
    kr, vr = tb.bitnet_kv4_read(c, *batch.tensors(DEV), m)
    new = 256
    batch = Batch([m], [new], 64)
    q = queries(new, heads, dim, "fp32") * 1e-3
    out, _ = run_attention(batch, c, q)
    off = []
    for h in range(0, heads, 11):
        z = q[:, h].double() @ kr[:, h].double().T * dim ** -0.5
        z.masked_fill_(torch.arange(m, device=DEV) > torch.arange(m - new, m, device=DEV)[:, None], -float("inf"))
        want = torch.softmax(z, -1) @ vr[:, h].double()
        off.append((out[:, h].double() - want) / want)
    off = torch.stack(off) / U
    most = 2 * m ** 0.5 + 32
    assert off.abs().max() <= most and off.mean().abs() <= most / 8, (off.abs().max(), off.mean(), most)
