"""The 4-bit paged KV cache on the GPU, against plain 64-bit arithmetic (kv4_ref.py).

Codes have to be those of the exact quantiser, everywhere; steps and values follow to their last roundings;
attention stays within bounds that count its roundings (kv4_ref.attention_bounds).  Memory that no row may reach
(unused pages, rows of nobody, places behind a sequence's end) is filled with rubbish and compared afterwards."""
import ctypes
import math

import pytest
import torch

import kv4_ref
import ternary_weight_bit_b200 as tb
from kv4_ref import U, Batch
from ternary_weight_bit_b200 import _native

pytestmark = pytest.mark.gpu

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert tb.bitnet_get_last_device_status() == 0, "a kernel recorded a status"


def rows_like_keys(shape, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    x = x * (3.0 / torch.randn((3, *shape[:-1], 1), generator=g).square().sum(0).clamp_min(0.05)).sqrt()
    x[..., ::16] *= 3.0
    return x


def rubbish_cache(pages, heads, dim, page, seed=0):
    """A cache full of rubbish: NaN and infinite steps, any codes."""
    g = torch.Generator(DEV).manual_seed(seed)
    c = tb.KV4Cache.empty(pages, heads, dim, page_size=page)
    for t in (c.k_codes, c.v_codes):
        t.random_(0, 256, generator=g)
    for t in (c.k_bos, c.v_bos):
        t.random_(-128, 128, generator=g)
    for t, bad in ((c.k_step, math.nan), (c.v_step, math.inf)):
        t.fill_(bad)
    return c


def copies(c):
    return {n: getattr(c, n).cpu().clone() for n in ("k_codes", "v_codes", "k_step", "v_step", "k_bos", "v_bos")}


def filled(batch, heads, dim, page, seed=0, bits=4):
    """A cache that bitnet_kv4_write has filled with every position of the batch's sequences, the rest rubbish, and
    the values it holds, as [(k, v)] per sequence in 64 bits."""
    c = rubbish_cache(batch.pages, heads, dim, page, seed)
    whole = Batch.__new__(Batch)
    whole.__dict__ = dict(batch.__dict__, new=batch.lens)
    whole.starts = torch.tensor([sum(batch.lens[:i]) for i in range(len(batch.lens) + 1)], dtype=torch.int32)
    T = int(whole.starts[-1])
    if T:
        k, v = (rows_like_keys((T, heads, dim), seed + s).to(DEV) for s in (1, 2))
        tb.bitnet_kv4_write(k, v, c, *whole.tensors(DEV), bits=bits)
    held = copies(c)
    return c, [tuple(kv4_ref.values(held[s + "_codes"], held[s + "_step"], held[s + "_bos"], batch, b) for s in "kv")
               for b in range(len(batch.lens))]


# ------------------------------------------------------------------ writing
def check_write(before, c, batch, k, v, bits, heads, dim):
    want = {n: t.clone() for n, t in before.items()}
    got = copies(c)
    places = list(batch.places())
    for side, x in (("k", k), ("v", v)):
        codes, step = kv4_ref.quantise(x.float(), bits)
        codes8, step8 = kv4_ref.quantise(x.float(), 8)
        for row, b, pos, page, off in places:
            if pos == 0:
                want[side + "_bos"][page] = codes8[row].to(torch.int8)
                want[side + "_codes"][page, :, off] = got[side + "_codes"][page, :, off]  # not read at position 0
            else:
                w = codes[row] & 15
                want[side + "_codes"][page, :, off] = (w[..., 0::2] | (w[..., 1::2] << 4)).to(torch.uint8)
            st = (step8 if pos == 0 else step)[row]
            g = got[side + "_step"][page, :, off].double()
            # 15 roundings: 7 + 5 additions, the mean's sum with eps, the division, one to spare
            assert ((g - st).abs() <= 15 * U * st).all()
            want[side + "_step"][page, :, off] = got[side + "_step"][page, :, off]
    for n in want:
        if n.endswith("step"):
            assert torch.equal(torch.nan_to_num(got[n], 7e37, 8e37), torch.nan_to_num(want[n], 7e37, 8e37)), n
        else:
            assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,new,heads,dim,page,bits", [
    ([1], [1], 1, 64, 16, 4),                           # the first token of all
    ([7], [1], 8, 128, 64, 4),
    ([130, 1, 64, 65, 0], [130, 1, 1, 65, 0], 3, 128, 64, 4),  # whole prompts, a page's last row, an empty sequence
    ([33, 200, 17], [16, 3, 17], 5, 64, 16, 3),
    ([300, 40], [299, 40], 2, 256, 32, 3),
    ([257], [256], 32, 128, 256, 4),
    ([5, 2], [9, 2], 2, 128, 16, 4),                    # more rows than positions: the first four are nowhere
    ([1200, 900, 333], [1200, 900, 333], 20, 128, 128, 4),  # several tokens to a CTA
])
def test_write(lens, new, heads, dim, page, bits, dtype):
    batch = Batch(lens, new, page, seed=dim + page, lead=2, tail=3)
    c = rubbish_cache(batch.pages, heads, dim, page)
    before = copies(c)
    k, v = (rows_like_keys((batch.rows, heads, dim), s).to(DTYPES[dtype]) for s in (3, 4))
    tb.bitnet_kv4_write(k.to(DEV), v.to(DEV), c, *batch.tensors(DEV), bits=bits)
    check_write(before, c, batch, k, v, bits, heads, dim)


def test_write_codes_next_to_a_border():
    # 3-bit rows with a maximum of 1: values around every half step, up to two fp32 steps to either side
    eps = float(torch.tensor(1e-5, dtype=torch.float32))
    mid = ((torch.arange(-3, 3).double() + 0.5) * (1.0 + eps) / 3.0).float()
    x = torch.zeros((64, 1, 64))
    for r in range(64):
        y = mid.clone()
        for _ in range(r % 3):
            y = torch.nextafter(y, torch.full_like(y, math.inf if r % 2 else -math.inf))
        x[r, 0, 1:7] = y
    x[..., 0] = 1.0
    batch = Batch([65], [64], 16)
    c = rubbish_cache(batch.pages, 1, 64, 16)
    before = copies(c)
    tb.bitnet_kv4_write(x.to(DEV), x.to(DEV), c, *batch.tensors(DEV), bits=3)
    check_write(before, c, batch, x, x, 3, 1, 64)


def test_write_of_many_rows_has_the_exact_codes():
    # 6 million values: a quantiser that decides in fp32 alone has some codes wrong here
    batch = Batch([6001, 5000], [6000, 4999], 64)
    x = rows_like_keys((batch.rows, 4, 128), 11)
    c = tb.KV4Cache.empty(batch.pages, 4, 128)
    tb.bitnet_kv4_write(x.to(DEV), -x.to(DEV), c, *batch.tensors(DEV))
    codes, _ = kv4_ref.quantise(x.to(DEV), 4)
    k, v = tb.bitnet_kv4_read(c, *batch.tensors(DEV), batch.rows)
    place = torch.tensor(list(batch.places()), device=DEV)
    for y, side, sign in ((k, "k", 1), (v, "v", -1)):
        step = getattr(c, side + "_step")[place[:, 3], :, place[:, 4]]
        want = (sign * codes[place[:, 0]]).clamp(-8, 7)
        if side == "v":
            want = kv4_ref.quantise(-x.to(DEV), 4)[0][place[:, 0]]
        assert torch.equal(y[place[:, 0]], step[..., None] * want.float())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads,dim,page,bits", [(1, 64, 16, 4), (1, 128, 64, 3), (3, 128, 16, 4), (2, 256, 64, 4), (3, 64, 256, 3), (1, 256, 32, 3)])
def test_many_rows_of_few_heads_are_those_of_more_heads(heads, dim, page, bits, dtype):
    """Many rows of few heads take another path of the kernels than the same rows among 16 heads."""
    batch = Batch([30000, 29000, 3000], [30000, 27001, 2500], page, lead=5, tail=9)
    k, v = (rows_like_keys((batch.rows, 16, dim), s).to(DTYPES[dtype]).to(DEV) for s in (1, 2))
    few, more = (rubbish_cache(batch.pages, h, dim, page) for h in (heads, 16))
    tensors = batch.tensors(DEV)
    for n in ("k_codes", "v_codes", "k_bos", "v_bos"):
        getattr(few, n).copy_(getattr(more, n)[:, :heads])  # the same rubbish
    tb.bitnet_kv4_write(k[:, :heads], v[:, :heads], few, *tensors, bits=bits)
    tb.bitnet_kv4_write(k, v, more, *tensors, bits=bits)
    for n, t in copies(few).items():
        same = getattr(more, n)[:, :heads].cpu()
        assert torch.equal(torch.nan_to_num(t.float(), 7e37, 8e37), torch.nan_to_num(same.float(), 7e37, 8e37)), n
    outs = []
    for c, h in ((few, heads), (more, 16)):
        out = [torch.full((batch.rows, h, dim), 123.0, dtype=DTYPES[dtype], device=DEV) for _ in range(2)]
        tb.bitnet_kv4_read(c, *tensors, batch.rows, dtype=DTYPES[dtype], k_out=out[0], v_out=out[1])
        outs.append(out)
    for a, b in zip(*outs):
        assert torch.equal(a, b[:, :heads]) and (a[:5] == 123.0).all() and (a[-9:] == 123.0).all()


@pytest.mark.parametrize("scale", [1e-38, 1e-20, 1e18, 2e36])
def test_write_of_tiny_and_huge_rows(scale):
    x = rows_like_keys((20, 2, 128), 5) * scale
    batch = Batch([20], [20], 16)
    c = rubbish_cache(batch.pages, 2, 128, 16)
    before = copies(c)
    tb.bitnet_kv4_write(x.to(DEV), x.to(DEV), c, *batch.tensors(DEV))
    check_write(before, c, batch, x, x, 4, 2, 128)


def test_rows_that_are_not_finite_stay_so():
    x = rows_like_keys((6, 1, 128), 5)
    x[2, 0, 7], x[3, 0, 9], x[4, 0, 3] = math.nan, math.inf, -math.inf
    for bits in (3, 4):
        batch = Batch([7], [6], 16)
        c = tb.KV4Cache.empty(batch.pages, 1, 128, page_size=16)
        tb.bitnet_kv4_write(x.to(DEV), x.to(DEV), c, *batch.tensors(DEV), bits=bits)
        k, _ = tb.bitnet_kv4_read(c, *batch.tensors(DEV), 6)
        fine = torch.isfinite(k).all(-1).all(-1).cpu()
        assert fine.tolist() == [True, True, False, False, False, True]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_write_takes_strided_rows_and_pieces(dtype):
    # keys and values as slices of one fused projection; the same rows at once, in two pieces, and one by one
    heads, dim, page, m = 5, 128, 16, 37
    fused = rows_like_keys((m, heads, 3, dim), 9).to(DTYPES[dtype]).to(DEV)
    k, v = fused[:, :, 1], fused[:, :, 2]
    whole = Batch([m], [m], page)
    c0 = rubbish_cache(whole.pages, heads, dim, page)
    tb.bitnet_kv4_write(k.contiguous(), v.contiguous(), c0, *whole.tensors(DEV))
    for cuts in ([0, m], [0, 16, m], list(range(m + 1))):
        c = rubbish_cache(whole.pages, heads, dim, page)
        for a, b in zip(cuts, cuts[1:]):
            part = Batch([b], [b - a], page)
            part.table, part.width = whole.table, whole.width
            tb.bitnet_kv4_write(k[a:b], v[a:b], c, *part.tensors(DEV))
        for n, t in copies(c0).items():
            assert torch.equal(torch.nan_to_num(copies(c)[n].double(), 1e300), torch.nan_to_num(t.double(), 1e300)), n


# ------------------------------------------------------------------ reading
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,new,heads,dim,page", [
    ([1], [1], 1, 64, 16),
    ([333], [333], 5, 128, 16),
    ([70, 0, 5, 129], [70, 0, 9, 2], 3, 256, 64),
    ([600, 700, 800], [600, 650, 1], 16, 64, 32),
])
def test_read(lens, new, heads, dim, page, dtype):
    batch = Batch(lens, new, page, seed=1, lead=1, tail=2)
    c, held = filled(batch, heads, dim, page)
    before = copies(c)
    k, v = (torch.full((batch.rows, heads, dim), 123.0, dtype=DTYPES[dtype], device=DEV) for _ in range(2))
    tb.bitnet_kv4_read(c, *batch.tensors(DEV), batch.rows, dtype=DTYPES[dtype], k_out=k, v_out=v)
    for side, y in enumerate((k, v)):
        want = torch.full((batch.rows, heads, dim), 123.0, dtype=torch.float64)
        want[int(batch.starts[0]):int(batch.starts[-1])] = 0.0  # rows before position 0
        for row, b, pos, _, _ in batch.places():
            want[row] = held[b][side][pos]
        assert torch.equal(y.cpu(), want.float().to(DTYPES[dtype]))
    after = copies(c)
    for n in before:
        assert torch.equal(torch.nan_to_num(after[n].double(), 1e300), torch.nan_to_num(before[n].double(), 1e300))


def test_read_one_side_only():
    batch = Batch([9], [9], 16)
    c, held = filled(batch, 2, 64, 16)
    v = torch.empty((9, 2, 64), device=DEV)
    tensors = batch.tensors(DEV)
    args = _native.Kv4Batch(*(t.data_ptr() for t in tensors), batch.width, 1, batch.width)
    assert _native.load().bitnet_kv4_read(c._ref, ctypes.byref(args), 9, None, v.data_ptr(), 0, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(v.cpu().double(), held[0][1].float().double())


# ------------------------------------------------------------------ attention
def largest(v):
    return float(v.abs().max()) if v.numel() else 0.0


def check_attention(batch, c, held, q, out, lse, scale, causal, window, untouched=123.0):
    dim, dtype = q.shape[-1], q.dtype
    assert out.dtype == dtype
    out, lse = out.cpu().double(), lse.cpu().double()
    mine = torch.zeros(batch.rows, dtype=torch.bool)
    for b in range(len(batch.lens)):
        s, e = int(batch.starts[b]), int(batch.starts[b + 1])
        mine[s:e] = True
        k, v = held[b]
        for i in range(s, e, 256):
            j = min(e, i + 256)
            m = batch.lens[b] - (e - j)  # positions up to the last of these rows
            kk, vv = (k, v) if not causal else (k[:max(m, 0)], v[:max(m, 0)])
            want, wl, top, mass = kv4_ref.attention(q[i:j].cpu().float(), kk, vv, scale, causal, window)
            err, lerr = kv4_ref.attention_bounds(want, top, mass, dim, kk.shape[0], dtype, largest(vv))
            off = (out[i:j] - want).abs()
            assert (off <= err).all(), f"sequence {b} rows {i - s}: off by {float((off / err).max()):.3g} times the bound"
            gone = wl == -math.inf
            assert torch.equal(lse[i:j] == -math.inf, gone)
            assert ((lse[i:j] - wl).abs()[~gone] <= (lerr + U * wl.abs() + 1e-30)[~gone]).all()
    assert (out[~mine] == untouched).all() and (lse[~mine] == untouched).all()


def run_attention(batch, c, q, scale=None, causal=True, window=0, max_q=0, **kw):
    out = torch.full(q.shape, 123.0, dtype=q.dtype, device=DEV)
    lse = torch.full(q.shape[:2], 123.0, device=DEV)
    tb.bitnet_kv4_attention(q, c, *batch.tensors(DEV), scale=scale, causal=causal, window=window, max_q=max_q,
                            return_lse=True, out=out, lse=lse, **kw)
    return out, lse


def queries(rows, heads, dim, dtype, seed=7):
    return torch.randn((rows, heads, dim), generator=torch.Generator().manual_seed(seed)).to(DTYPES[dtype]).to(DEV)


SHAPES = [
    # lens, new, heads, kv heads, dim, page
    ([1], [1], 1, 1, 64, 16),
    ([2], [2], 8, 8, 128, 64),
    ([500], [1], 32, 8, 128, 64),
    ([31, 32, 33, 64, 65, 1, 127, 129], [1] * 8, 12, 4, 128, 16),
    ([17, 100, 300], [1, 1, 1], 5, 1, 256, 32),
    ([700, 0, 40, 5000], [1, 0, 1, 1], 16, 2, 64, 16),          # an empty sequence between others
    ([0, 3], [2, 5], 4, 2, 128, 16),                            # rows that stand before the cache
    ([90, 257, 12], [3, 6, 2], 40, 8, 64, 32),                  # draft tokens
    ([64, 600], [64, 17], 6, 2, 128, 128),
    ([300, 129, 7], [300, 128, 7], 8, 2, 128, 64),              # prompts
    ([515], [515], 3, 3, 64, 256),
    ([1000, 260], [130, 1], 24, 3, 256, 64),                    # a chunk beside a step
    ([4100, 2000, 2048, 70], [1, 1, 1, 1], 64, 1, 128, 64),     # 64 query heads of one key head
    ([20000], [1], 8, 8, 128, 64),                              # long
    ([9000, 37], [1, 30], 7, 7, 64, 64),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,new,heads,kv,dim,page", SHAPES)
def test_attention(lens, new, heads, kv, dim, page, dtype):
    batch = Batch(lens, new, page, seed=kv, lead=1, tail=2)
    c, held = filled(batch, kv, dim, page, bits=3 if kv == 3 else 4)
    q = queries(batch.rows, heads, dim, dtype)
    for max_q in {0, max(new)}:
        out, lse = run_attention(batch, c, q, max_q=max_q)
        check_attention(batch, c, held, q, out, lse, dim ** -0.5, True, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("window", [1, 2, 31, 64, 100, 5000, 1 << 40])
@pytest.mark.parametrize("lens,new,heads,kv,dim,page", [
    ([400, 70, 1], [1, 1, 1], 8, 2, 128, 16),
    ([333, 64], [40, 64], 16, 2, 64, 64),
    ([260], [260], 4, 4, 128, 64),
    ([70], [33], 2, 1, 256, 32),
])
def test_attention_window(lens, new, heads, kv, dim, page, window, dtype):
    batch = Batch(lens, new, page, lead=1, tail=1)
    c, held = filled(batch, kv, dim, page)
    for b in range(len(lens)):  # pages behind every window may be gone
        first = max(0, lens[b] - new[b] - window + 1) // page
        batch.table[b, :first] = -7
    q = queries(batch.rows, heads, dim, dtype)
    out, lse = run_attention(batch, c, q, window=window)
    check_attention(batch, c, held, q, out, lse, dim ** -0.5, True, window)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,new,heads,kv,dim,page", [
    ([50, 0, 200], [1, 2, 9], 8, 2, 128, 16),
    ([130, 20], [200, 64], 4, 4, 64, 64),     # more queries than positions: all are seen
    ([1, 65], [70, 140], 2, 2, 128, 32),
    ([90], [40], 3, 1, 256, 16),
])
def test_attention_without_a_causal_mask(lens, new, heads, kv, dim, page, dtype):
    batch = Batch(lens, new, page, lead=1, tail=1)
    c, held = filled(batch, kv, dim, page)
    q = queries(batch.rows, heads, dim, dtype)
    out, lse = run_attention(batch, c, q, causal=False, scale=0.3)
    check_attention(batch, c, held, q, out, lse, 0.3, False, 0)


@pytest.mark.parametrize("new", [1, 40, 200])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_of_large_small_and_zero_queries(dtype, new):
    batch = Batch([300], [new], 64)
    c, held = filled(batch, 2, 128, 64)
    for size, scale in ((1e4, None), (1e-30, None), (0.0, None), (1e30, 1e-31), (1e-3, -50.0), (1.0, 0.0)):
        q = queries(batch.rows, 4, 128, dtype) * size
        scale = 128 ** -0.5 if scale is None else scale
        out, lse = run_attention(batch, c, q, scale=scale)
        check_attention(batch, c, held, q, out, lse, scale, True, 0)


@pytest.mark.parametrize("new", [1, 40, 200])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_of_rows_with_steps_far_apart(dtype, new):
    # values of very different sizes in one cache, the largest first, last or in the middle
    for turn in (0, 1, 2):
        batch = Batch([260], [260], 64)
        size = torch.logspace(-6, 6, 260)
        size = (size, size.flip(0), torch.cat((size[130:], size[:130])))[turn][:, None, None]
        k, v = rows_like_keys((260, 2, 128), 21), rows_like_keys((260, 2, 128), 22) * size
        c = rubbish_cache(batch.pages, 2, 128, 64)
        tb.bitnet_kv4_write(k.to(DEV), v.to(DEV), c, *batch.tensors(DEV))
        held = copies(c)
        batch = Batch([260], [new], 64)
        held = [tuple(kv4_ref.values(held[s + "_codes"], held[s + "_step"], held[s + "_bos"], batch, 0) for s in "kv")]
        q = queries(new, 4, 128, dtype)
        out, lse = run_attention(batch, c, q)
        check_attention(batch, c, held, q, out, lse, 128 ** -0.5, True, 0)


@pytest.mark.parametrize("new", [1, 60, 300])
def test_a_query_that_is_not_finite_keeps_to_its_row(new):
    batch = Batch([400, 50], [new, 1], 64)
    c, held = filled(batch, 2, 128, 64)
    for dtype in ("bf16", "fp32"):
        q = queries(batch.rows, 8, 128, dtype)
        good, _ = run_attention(batch, c, q)
        bad = q.clone()
        bad[0, 3, 5], bad[batch.rows - 1, 6, 0] = math.nan, math.inf
        out, _ = run_attention(batch, c, bad)
        assert torch.isnan(out[0, 3]).all() and not torch.isfinite(out[batch.rows - 1, 6]).any()
        keep = torch.ones(q.shape[:2], dtype=torch.bool, device=DEV)
        keep[0, 3] = keep[batch.rows - 1, 6] = False
        assert torch.equal(out[keep], good[keep])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [0, 1, 3, 70])
def test_one_sequence_with_few_of_many_rows(new, dim, dtype):
    batch = Batch([max(new, 300)], [new], 32, lead=30, tail=200)
    c, held = filled(batch, 2, dim, 32)
    q = queries(batch.rows, 8, dim, dtype)
    out, lse = run_attention(batch, c, q)
    check_attention(batch, c, held, q, out, lse, dim ** -0.5, True, 0)


@pytest.mark.parametrize("new", [1, 30, 200])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pos", [0, 5, 250])
def test_a_step_that_is_not_finite_keeps_to_the_rows_that_see_it(pos, dtype, new):
    batch = Batch([300], [new], 64)
    c, _ = filled(batch, 2, 128, 64)
    q = queries(new, 4, 128, dtype)
    for window in (0, 60):
        want, _ = run_attention(batch, c, q, window=window)
        for side, bad in (("v_step", math.inf), ("v_step", math.nan), ("k_step", math.nan)):
            step = getattr(c, side)[int(batch.table[0, pos // 64]), 1]
            kept = step[pos % 64].clone()
            step[pos % 64] = bad
            got, _ = run_attention(batch, c, q, window=window)
            step[pos % 64] = kept
            at = torch.arange(300 - new, 300)
            sees = (at >= pos) & ((at - pos < window) | (window == 0))
            assert got[sees.to(DEV), 2:].isnan().all()
            assert torch.equal(got[:, :2], want[:, :2]) and torch.equal(got[~sees.to(DEV)], want[~sees.to(DEV)])


@pytest.mark.parametrize("new", [1, 50, 200])
def test_attention_takes_strided_queries_and_gives_equal_bits(new):
    batch = Batch([333, 90], [new, 3], 16)
    c, held = filled(batch, 4, 64, 16)
    for dtype in ("bf16", "fp32"):
        fused = torch.randn((batch.rows, 3, 12, 64), device=DEV).to(DTYPES[dtype])
        want = run_attention(batch, c, fused[:, 1].contiguous())
        for _ in range(3):
            got = run_attention(batch, c, fused[:, 1])
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        # head-major memory
        turned = fused[:, 1].transpose(0, 1).contiguous().transpose(0, 1)
        got = run_attention(batch, c, turned)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_over_a_cache_past_32_bits():
    # 5 GB of codes to a side: the pages in use lie at its far end
    pages, heads, page, dim = 160000, 8, 64, 128
    assert pages * heads * page * dim // 2 > 2 ** 32
    c = tb.KV4Cache.empty(pages, heads, dim, page_size=page)
    batch = Batch([200, 77], [200, 77], page, first_page=pages - 9)
    assert int(batch.table.max()) < pages
    k, v = (rows_like_keys((batch.rows, heads, dim), s).to(DEV) for s in (1, 2))
    tb.bitnet_kv4_write(k, v, c, *batch.tensors(DEV))
    kr, vr = tb.bitnet_kv4_read(c, *batch.tensors(DEV), batch.rows)
    held = [(kr[a:b].cpu().double(), vr[a:b].cpu().double()) for a, b in ((0, 200), (200, 277))]
    for x, y in ((k, kr), (v, vr)):
        codes, step = kv4_ref.quantise(x, 4)
        want = codes[1:200] * step[1:200, :, None]
        assert ((y[1:200].double() - want).abs() <= 17 * U * want.abs()).all()
    for new in ([1, 1], [200, 77]):
        b2 = Batch([200, 77], new, page, first_page=pages - 9)
        for dtype in ("bf16", "fp32"):
            q = queries(b2.rows, 16, dim, dtype)
            out, lse = run_attention(b2, c, q)
            check_attention(b2, c, held, q, out, lse, dim ** -0.5, True, 0)


@pytest.mark.parametrize("new", [1, 40, 150])
def test_bad_pages_and_lengths_are_recorded_and_left_out(new):
    # page numbers outside the cache and a length past the table: no access, a status, the rest as without them
    batch = Batch([200], [new], 16)
    c, held = filled(batch, 2, 128, 16)
    q = queries(new, 4, 128, "fp32")
    table, lens, starts = batch.tensors(DEV)
    bad = table.clone()
    bad[0, 3], bad[0, 5] = -1, batch.pages
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    tb.bitnet_kv4_attention(q, c, bad, lens, starts, out=out, lse=lse)
    assert tb.bitnet_get_last_device_status() == _native.ERR_INVALID_ARG
    gone = torch.zeros(200, dtype=torch.bool)
    gone[48:64] = gone[80:96] = True
    k, v = held[0]
    scale = 128 ** -0.5
    for i in range(new):
        seen = ~gone[:200 - new + i + 1]
        want, _, top, mass = kv4_ref.attention(q[i:i + 1].cpu(), k[:len(seen)][seen], v[:len(seen)][seen], scale, True, 0)
        err, _ = kv4_ref.attention_bounds(want, top, mass, 128, 200, torch.float32, largest(v))
        assert ((out[i:i + 1].cpu().double() - want).abs() <= err).all()
    tb.bitnet_kv4_attention(q, c, table, lens + 1000, starts, causal=False, out=out)
    assert tb.bitnet_get_last_device_status() == _native.ERR_INVALID_ARG
    before = copies(c)
    rows = rows_like_keys((new, 2, 128), 3).to(DEV)
    tb.bitnet_kv4_write(rows, rows, c, bad.fill_(batch.pages), lens, starts)
    assert tb.bitnet_get_last_device_status() == _native.ERR_INVALID_ARG
    for n, t in copies(c).items():
        assert torch.equal(torch.nan_to_num(t.double(), 1e300), torch.nan_to_num(before[n].double(), 1e300))
    kr, vr = tb.bitnet_kv4_read(c, bad, lens, starts, new)
    assert tb.bitnet_get_last_device_status() == _native.ERR_INVALID_ARG
    assert not kr.any() and not vr.any()


def test_rows_past_the_tensor_are_not_touched():
    # q_starts that promise more rows than the tensors have (another T may split the work in another way)
    batch = Batch([100, 50], [60, 50], 16)
    c, held = filled(batch, 2, 64, 16)
    q = queries(batch.rows, 2, 64, "bf16")
    whole, wl = run_attention(batch, c, q)
    for T in (1, 30, 61, 90):
        big = torch.full((batch.rows, 2, 64), 123.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((batch.rows, 2), 123.0, device=DEV)
        tb.bitnet_kv4_attention(q[:T], c, *batch.tensors(DEV), out=big[:T], lse=lse[:T])
        assert (big[T:] == 123.0).all() and (lse[T:] == 123.0).all()
        big[T:], lse[T:] = whole[T:], wl[T:]
        check_attention(batch, c, held, q, big, lse, 64 ** -0.5, True, 0)


def test_streams_and_captured_graphs():
    # two attentions at once on streams of their own, and a captured step (write, then attend) replayed on new inputs
    batch = Batch([700, 90, 1500], [1, 1, 1], 64)
    c, held = filled(batch, 4, 128, 64)
    q = [queries(3, 16, 128, "bf16", seed=s) for s in (1, 2)]
    want = [run_attention(batch, c, x) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in q]
    got = []
    for _ in range(5):
        got = []
        for x, s in zip(q, streams):
            with torch.cuda.stream(s):
                got.append(run_attention(batch, c, x))
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)
    # a stream given by argument
    out = torch.empty_like(q[0])
    ws = torch.empty(tb.bitnet_kv4_attention_workspace_bytes(3, 16, 4, 128, 3), dtype=torch.uint8, device=DEV)
    tensors = batch.tensors(DEV)
    torch.cuda.synchronize()
    tb.bitnet_kv4_attention(q[1], c, *tensors, out=out, ws=ws, stream=streams[0])
    torch.cuda.synchronize()
    assert torch.equal(out, want[1][0])

    table, lens, starts = batch.tensors(DEV)
    k, v, x = (torch.zeros((3, h, 128), dtype=torch.bfloat16, device=DEV) for h in (4, 4, 16))
    graph = torch.cuda.CUDAGraph()
    tb.bitnet_kv4_write(k, v, c, table, lens, starts)
    with torch.cuda.graph(graph):
        tb.bitnet_kv4_write(k, v, c, table, lens, starts)
        res = tb.bitnet_kv4_attention(x, c, table, lens, starts, ws=ws, out=out)
    for step in range(3):
        nk, nv = (rows_like_keys((3, 4, 128), 30 + 2 * step + i).to(torch.bfloat16).to(DEV) for i in (0, 1))
        nx = queries(3, 16, 128, "bf16", seed=50 + step)
        k.copy_(nk), v.copy_(nv), x.copy_(nx)
        graph.replay()
        replayed = res.clone()
        tb.bitnet_kv4_write(nk, nv, c, table, lens, starts)
        assert torch.equal(replayed, tb.bitnet_kv4_attention(nx, c, table, lens, starts))
        lens += 1  # the graph follows the lengths; every last page has room


def test_memory_of_a_call_comes_from_its_stream():
    batch = Batch([300, 40], [1, 3], 64, seed=5)
    c, _ = filled(batch, 2, 64, 64, seed=5)
    q = queries(4, 4, 64, "bf16", seed=5)
    tensors = batch.tensors(DEV)
    want = tb.bitnet_kv4_attention(q, c, *tensors, return_lse=True) + tb.bitnet_kv4_read(c, *tensors, 4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda.memory._record_memory_history(context=None, max_entries=100)
    got = tb.bitnet_kv4_attention(q, c, *tensors, return_lse=True, stream=side) + tb.bitnet_kv4_read(c, *tensors, 4, stream=side)
    traces = torch.cuda.memory._snapshot()["device_traces"][torch.cuda.current_device()]
    torch.cuda.memory._record_memory_history(enabled=None)
    streams = [e["stream"] for e in traces if e["action"] == "alloc"]
    assert streams == [side.cuda_stream] * 5  # output, sums and workspace; keys and values
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_rows_and_no_sequences():
    batch = Batch([5], [0], 16)
    c, _ = filled(batch, 1, 64, 16)
    q = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    assert tb.bitnet_kv4_attention(q, c, *batch.tensors(DEV)).shape == (0, 2, 64)
    none = (torch.empty((0, 4), dtype=torch.int32, device=DEV), torch.empty((0,), dtype=torch.int32, device=DEV),
            torch.zeros((1,), dtype=torch.int32, device=DEV))
    out = torch.full((3, 2, 64), 5.0, device=DEV)
    tb.bitnet_kv4_attention(torch.zeros((3, 2, 64), device=DEV), c, *none, out=out)
    assert (out == 5.0).all()
    k, v = tb.bitnet_kv4_read(c, *batch.tensors(DEV), 0)
    assert k.shape == (0, 1, 64)
    # sequences of which none has a row, for rows of nobody
    out = torch.full((3, 2, 64), 5.0, device=DEV)
    tb.bitnet_kv4_attention(torch.zeros((3, 2, 64), device=DEV), c, *batch.tensors(DEV), out=out)
    assert (out == 5.0).all()


def test_many_sequences():
    lens = [(37 * i) % 211 for i in range(700)]
    batch = Batch(lens, [min(1, m) for m in lens], 16)
    c, held = filled(batch, 1, 64, 16)
    q = queries(batch.rows, 4, 64, "bf16")
    out, lse = run_attention(batch, c, q, max_q=1)
    check_attention(batch, c, held, q, out, lse, 64 ** -0.5, True, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("width", [8, 9, 16, 17, 90])  # whether items are shared between CTAs goes by the table's width
def test_short_contexts_with_narrow_and_wide_tables(width, dtype):
    lens = [(61 * i) % 500 + 3 for i in range(50)]
    for sequences in (2, 50):
        batch = Batch(lens[:sequences], [1 + i % 3 for i in range(sequences)], 64, width=width)
        c, held = filled(batch, 8, 128, 64)
        q = queries(batch.rows, 8, 128, dtype)
        out, lse = run_attention(batch, c, q, max_q=3)
        check_attention(batch, c, held, q, out, lse, 128 ** -0.5, True, 0)


# ------------------------------------------------------------------ together, as a layer uses them
def test_an_attention_layer_prefills_and_decodes():
    """Wq, Wk, Wv (ternary, H-BitLinear) -> cache -> attention -> Wo: a prompt at once and then token by token, against
    the same layer in 64 bits on the cached values, and against the whole sequence at once."""
    hidden, heads, kv, dim, page = 512, 8, 2, 64, 16
    g = torch.Generator().manual_seed(3)
    mats = {n: torch.randn((r, hidden), generator=g) * 0.02 for n, r in
            (("q", heads * dim), ("k", kv * dim), ("v", kv * dim), ("o", hidden))}
    layer = {n: tb.HBitLinear(w.to(DEV), mode="int8", fwht=n == "o") for n, w in mats.items()}
    x = torch.randn((2, 45, hidden), generator=g).to(DEV)
    prompts, steps = [21, 33], 12

    def project(rows):
        return [layer[n](rows).view(rows.shape[0], -1, dim) for n in "qkv"]

    def forward(cache, batch, rows):
        q, k, v = project(rows)
        where = batch.tensors(DEV)
        tb.bitnet_kv4_write(k, v, cache, *where)
        a = tb.bitnet_kv4_attention(q, cache, *where)
        return a, layer["o"](a.reshape(rows.shape[0], -1))

    def place(lens, new):
        batch = Batch(lens, new, page)
        batch.table = torch.tensor([[0, 4, 2, 8], [3, 1, 7, 6]], dtype=torch.int32)
        return batch

    cache = rubbish_cache(9, kv, dim, page)
    outs = [[], []]
    a, y = forward(cache, place(prompts, prompts), torch.cat([x[b, :n] for b, n in enumerate(prompts)]))
    for b, part in enumerate(y.split(prompts)):
        outs[b].append(part)
    for i in range(steps):
        lens = [n + i + 1 for n in prompts]
        a, y = forward(cache, place(lens, [1, 1]), torch.stack([x[b, m - 1] for b, m in enumerate(lens)]))
        outs[0].append(y[:1]), outs[1].append(y[1:])
    # the last step's attention against 64 bits on what the cache holds
    last = place(lens, [1, 1])
    held = copies(cache)
    for b in range(2):
        k, v = (kv4_ref.values(held[s + "_codes"], held[s + "_step"], held[s + "_bos"], last, b) for s in "kv")
        q = project(x[b, lens[b] - 1][None])[0]
        want, _, top, mass = kv4_ref.attention(q.cpu(), k, v, dim ** -0.5, True, 0)
        err, _ = kv4_ref.attention_bounds(want, top, mass, dim, lens[b], torch.float32, largest(v))
        assert ((a[b].cpu().double() - want[0]).abs() <= err[0]).all()
    # the whole at once: the same cache bytes, and outputs that differ by roundings (a code may flip in Wo's quantiser:
    # one step of int8 in one of 512 inputs moves an output by at most max|a| / 127 * alpha)
    other = rubbish_cache(9, kv, dim, page)
    whole = place(lens, lens)
    a, y = forward(other, whole, torch.cat([x[b, :m] for b, m in enumerate(lens)]))
    for n, t in copies(other).items():
        assert torch.equal(torch.nan_to_num(t.double(), 1e300), torch.nan_to_num(held[n].double(), 1e300)), n
    for b, part in enumerate(y.split(lens)):
        got = torch.cat(outs[b])
        assert (got - part).abs().max() <= 0.02 * part.abs().max()
