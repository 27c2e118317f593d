"""The 4-bit paged KV cache on the host: which calls its C entry points and its binding refuse, before any CUDA
work, and the plain implementation that the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import kv4_ref
import ternary_weight_bit_b200 as tb
from ternary_weight_bit_b200 import _native

P = ctypes.c_void_p
FAKE = P(1 << 20)  # aligned, never dereferenced: every call below is refused or empty
BAD = _native.ERR_INVALID_ARG
SHAPE = _native.ERR_UNSUPPORTED_SHAPE


@pytest.fixture(scope="module")
def L():
    return _native.load()


def cache(**kw):
    c = {n: 1 << 20 for n in ("k_codes", "v_codes", "k_step", "v_step", "k_bos", "v_bos")}
    c.update(pages=8, heads=4, page_size=64, dim=128)
    c.update(kw)
    return ctypes.byref(_native.Kv4Cache(**c))


def batch(**kw):
    b = dict(block_table=1 << 20, kv_lens=1 << 20, q_starts=1 << 20, table_stride=3, batch=2, max_pages=3)
    b.update(kw)
    return ctypes.byref(_native.Kv4Batch(**b))


BAD_CACHES = [(dict(dim=96), SHAPE), (dict(dim=0), SHAPE), (dict(page_size=48), SHAPE), (dict(page_size=8), SHAPE),
              (dict(page_size=512), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=-64), SHAPE),
              (dict(heads=0), SHAPE), (dict(heads=1 << 16), SHAPE), (dict(pages=-1), BAD), (dict(pages=1 << 32), BAD),
              (dict(k_codes=None), BAD), (dict(v_codes=(1 << 20) + 8), BAD), (dict(k_step=None), BAD),
              (dict(v_step=(1 << 20) + 4), BAD), (dict(k_bos=None), BAD), (dict(v_bos=(1 << 20) + 1), BAD)]
BAD_BATCHES = [(dict(batch=-1), BAD), (dict(batch=1 << 16), BAD), (dict(max_pages=-1), BAD), (dict(table_stride=2), BAD),
               (dict(block_table=None), BAD), (dict(kv_lens=None), BAD), (dict(q_starts=None), BAD),
               (dict(kv_lens=(1 << 20) + 2), BAD)]


def write(L, T=5, k=FAKE, v=FAKE, dt=1, ks=(512, 128), vs=(512, 128), c=None, b=None, bits=4, eps=1e-5):
    return L.bitnet_kv4_write(k, v, dt, T, *ks, *vs, c or cache(), b or batch(), bits, eps, P(0))


def read(L, T=5, k=FAKE, v=FAKE, dt=0, c=None, b=None):
    return L.bitnet_kv4_read(c or cache(), b or batch(), T, k, v, dt, P(0))


def attend(L, T=5, q=FAKE, dt=1, heads=8, qs=(1024, 128), c=None, b=None, scale=0.1, causal=1, window=0, max_q=0, out=FAKE,
           lse=None, ws=FAKE, nws=1 << 40):
    return L.bitnet_kv4_attention(q, dt, T, heads, *qs, c or cache(), b or batch(), scale, causal, window, max_q, out, lse,
                                  ws, nws, P(0))


@pytest.mark.parametrize("call", [write, read, attend])
def test_refused_caches_and_batches(L, call):
    for kw, want in BAD_CACHES:
        assert call(L, c=cache(**kw)) == want, kw
    for kw, want in BAD_BATCHES:
        assert call(L, b=batch(**kw)) == want, kw
    assert call(L, T=-1) == BAD and call(L, T=(1 << 30) + 1) == BAD
    assert call(L, dt=2) == BAD and call(L, dt=-1) == BAD
    # nothing to do: no rows, or no sequences
    assert call(L, T=0) == _native.OK
    assert call(L, b=batch(batch=0)) == _native.OK
    assert call(L, T=0, c=cache(dim=96)) == SHAPE


def test_refused_writes(L):
    for kw in (dict(bits=8), dict(bits=0), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf),
               dict(k=None), dict(v=None), dict(k=P((1 << 20) + 8)), dict(v=P((1 << 20) + 2)), dict(ks=(516, 128)),
               dict(ks=(512, 4)), dict(vs=(-512, 128)), dict(vs=(512, -8)), dict(vs=(1 << 40, 128)),
               dict(dt=0, ks=(512, 130))):
        assert write(L, **kw) == BAD, kw


def test_refused_reads(L):
    assert read(L, k=P((1 << 20) + 8)) == BAD and read(L, v=P((1 << 20) + 4)) == BAD
    assert read(L, k=None, v=None) == _native.OK  # nothing asked for


def test_refused_attention(L):
    for kw in (dict(scale=math.nan), dict(scale=math.inf), dict(causal=2), dict(window=-1), dict(window=4, causal=0),
               dict(max_q=-1), dict(q=None), dict(q=P((1 << 20) + 8)), dict(out=None), dict(out=P((1 << 20) + 8)),
               dict(lse=P((1 << 20) + 2)), dict(qs=(1020, 128)), dict(qs=(1024, -128))):
        assert attend(L, **kw) == BAD, kw
    for heads in (0, 2, 6, 1 << 16, -4):
        assert attend(L, heads=heads) == SHAPE, heads
    # rows of all heads are counted in 31 bits
    assert attend(L, T=1 << 28) == SHAPE and L.bitnet_kv4_attention_workspace_bytes(1 << 28, 8, 4, 128, 2) == 0
    need = L.bitnet_kv4_attention_workspace_bytes(5, 8, 4, 128, 2)
    assert need > 0
    assert attend(L, ws=None, nws=0) == _native.ERR_WORKSPACE
    assert attend(L, nws=need - 1) == _native.ERR_WORKSPACE
    assert attend(L, ws=P((1 << 20) + 128)) == _native.ERR_WORKSPACE
    for sizes in ((0, 8, 4, 128, 2), (5, 6, 4, 128, 2), (5, 8, 4, 96, 2), (5, 8, 0, 128, 2), (5, 8, 4, 128, 0)):
        assert L.bitnet_kv4_attention_workspace_bytes(*sizes) == 0, sizes


def test_binding_refuses_cpu_tensors_and_wrong_types():
    codes = torch.zeros((2, 4, 64, 64), dtype=torch.uint8)
    step, bos = torch.zeros((2, 4, 64)), torch.zeros((2, 4, 128), dtype=torch.int8)
    with pytest.raises(ValueError, match="CUDA"):
        tb.KV4Cache(codes, codes, step, step, bos, bos)
    with pytest.raises(TypeError):
        tb.KV4Cache(None, codes, step, step, bos, bos)
    with pytest.raises(ValueError, match="even"):
        tb.KV4Cache.empty(1, 1, 63, device="cpu")
    i = torch.zeros((1,), dtype=torch.int32)
    for call in (lambda: tb.bitnet_kv4_write(step, step, "cache", i, i, i),
                 lambda: tb.bitnet_kv4_read("cache", i, i, i, 1),
                 lambda: tb.bitnet_kv4_attention(step, None, i, i, i)):
        with pytest.raises(TypeError, match="KV4Cache"):
            call()


# ------------------------------------------------------------------ the plain implementation
def test_plain_quantiser_on_hand_worked_rows():
    # mean|x| = 2, so a 4-bit step of (2 + 1e-5) / sqrt 7 = 0.7559: 4 -> 5.29, -4 -> -5.29, 0
    codes, step = kv4_ref.quantise(torch.tensor([4.0, -4.0, 0.0, 0.0]), 4)
    assert codes.tolist() == [5, -5, 0, 0] and abs(float(step) - 0.755933) < 1e-5
    codes, step = kv4_ref.quantise(torch.tensor([3.0, -3.0, 1.6, 0.4]), 3)
    assert codes.tolist() == [3, -3, 2, 0] and abs(float(step) - 1.0) < 1e-4
    codes, _ = kv4_ref.quantise(torch.tensor([100.0, 0.0, 0.0, 0.0]), 4)  # clipped
    assert codes.tolist() == [7, 0, 0, 0]


def test_plain_attention_on_hand_worked_rows():
    k = torch.tensor([[[1.0, 0.0]], [[0.0, 1.0]]], dtype=torch.float64)
    v = torch.tensor([[[2.0, 0.0]], [[0.0, 4.0]]], dtype=torch.float64)
    q = torch.tensor([[[math.log(3.0), 0.0]]])
    out, lse, _, _ = kv4_ref.attention(q, k, v, 1.0, True, 0)  # weights 3/4 and 1/4
    assert torch.allclose(out, torch.tensor([[[1.5, 1.0]]], dtype=torch.float64), atol=1e-7)
    assert abs(float(lse) - math.log(4.0)) < 1e-6
    out, lse, _, _ = kv4_ref.attention(q, k, v, 1.0, True, 1)  # the last position alone
    assert out.tolist() == [[[0.0, 4.0]]] and float(lse) == 0.0
    out, lse, _, _ = kv4_ref.attention(torch.ones((3, 1, 2)), k, v, 1.0, True, 0)  # the first row stands before the cache
    assert out[0].abs().sum() == 0 and float(lse[0, 0]) == -math.inf and out[1].tolist() == [[2.0, 0.0]]
