"""ternary_weight_bit_b200 -- the BitNet H-BitLinear forward path on B200 (sm_100a).

Python front end of libbitnet.so.  The functions carry the names of the C ABI
(include/bitnet.h) and only marshal arguments: torch tensors supply device
memory and the current CUDA stream, the kernels of libbitnet.so do every step.
There is no CPU or PyTorch fallback; a missing library or a non-CUDA tensor
raises.

    packed, alpha = bitnet_pack_ternary(W)                        # once per weight
    out = bitnet_hbitlinear_forward(X, packed, alpha, N, fwht=True, mode="int4")

The step-by-step entry points bitnet_act_quant and bitnet_ternary_gemm expose the
intermediate int8 codes, per-token scales and (optionally) the int32 accumulators.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _native
from ._native import BitnetError

__all__ = [
    "BitnetError", "HBitLinear", "bitnet_pack_ternary", "bitnet_act_quant", "bitnet_ternary_gemm",
    "bitnet_hbitlinear_forward", "bitnet_hbitlinear_forward_noalloc", "bitnet_forward_workspace_bytes", "bitnet_pack_workspace_bytes",
    "bitnet_get_last_device_status", "bitnet_selftest_wait_timeout", "bitnet_abi_version", "mode_id",
    "bitnet_gemm_token_tile", "bitnet_gemm_force_token_tile", "bitnet_gemm_force_k_splits",
    "bitnet_forward_gemm_plan", "bitnet_workspace_bytes", "bitnet_gemm_workspace_bytes",
    "bitnet_forward_kernel_count", "bitnet_tl2_bytes", "bitnet_pack_tl2", "bitnet_ternary_gemm_tl2",
    "bitnet_hbitlinear_forward_tl2",
    "bitnet_act_quant_swiglu", "bitnet_hbitlinear_forward_swiglu", "bitnet_kv_quant",
    "bitnet_ternary_gemm_ex", "bitnet_hbitlinear_forward_ex",
    "KV4Cache", "bitnet_kv4_write", "bitnet_kv4_read", "bitnet_kv4_attention", "bitnet_kv4_attention_workspace_bytes",
]

_MODES = {"int8": _native.ACT_INT8_ABSMAX, "int4": _native.ACT_INT4_ABSMEAN}


def mode_id(mode) -> int:
    if isinstance(mode, int):
        return mode
    try:
        return _MODES[mode]
    except KeyError:
        raise ValueError(f"mode must be 'int8' or 'int4', got {mode!r}") from None


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t: torch.Tensor, name: str, dtype=None, shape=None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libbitnet has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def bitnet_abi_version() -> int:
    return _native.load().bitnet_abi_version()


def bitnet_gemm_token_tile(M: int, N: int, K: int) -> int:
    """Token-tile size of the tcgen05 GEMM for this shape (0: decode kernel, -1: rejected)."""
    return _native.load().bitnet_gemm_token_tile(M, N, K)


def bitnet_forward_gemm_plan(M: int, N: int, K: int) -> tuple:
    """(token tile, k-splits) of the GEMM inside the forward; (0, 0) for the decode kernel."""
    sp = ctypes.c_int(0)
    tile = _native.load().bitnet_forward_gemm_plan(M, N, K, ctypes.byref(sp))
    return tile, sp.value


def bitnet_gemm_force_token_tile(token_tile: int) -> None:
    """Force the GEMM token tile (256/224/192/128/64) process-wide; 0 restores the automatic choice."""
    _native.check("bitnet_gemm_force_token_tile", _native.load().bitnet_gemm_force_token_tile(token_tile))


def bitnet_gemm_force_k_splits(k_splits: int) -> None:
    """Force the forward's k-split count (0 = automatic; 1, 2, 4, 8 where the shape allows it)."""
    _native.check("bitnet_gemm_force_k_splits", _native.load().bitnet_gemm_force_k_splits(k_splits))


def bitnet_pack_workspace_bytes(N: int, K: int) -> int:
    return _native.load().bitnet_pack_workspace_bytes(N, K)


def bitnet_workspace_bytes(M: int, N: int, K: int) -> int:
    """One workspace size that serves pack, forward and GEMM on an M x N x K problem."""
    return _native.load().bitnet_workspace_bytes(M, N, K)


def bitnet_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return _native.load().bitnet_gemm_workspace_bytes(M, N, K)


def bitnet_forward_kernel_count(M: int, N: int, K: int, fwht: bool = True, gain: bool = False) -> int:
    """Kernels the forward launches for this problem (1 when the decode kernel runs the
    activation step itself, else 2; 0 for M == 0; -1 for rejected sizes)."""
    return _native.load().bitnet_forward_kernel_count(M, N, K, int(bool(fwht)), int(bool(gain)))


def bitnet_forward_workspace_bytes(M: int, K: int) -> int:
    return _native.load().bitnet_forward_workspace_bytes(M, K)


def bitnet_pack_ternary(W: torch.Tensor, eps: float = 1e-5, packed=None, alpha=None, ws=None, stream=None):
    """Ternarise W [N, K] (fp32, CUDA) with its absmean and pack it at 2 bits per weight.

    Returns (packed uint8 [N, K/4], alpha float32 [1]), both on W's device."""
    L = _native.load()
    _need(W, "W", torch.float32)
    N, K = W.shape
    dev = W.device
    packed = torch.empty((N, K // 4), dtype=torch.uint8, device=dev) if packed is None else packed
    alpha = torch.empty((1,), dtype=torch.float32, device=dev) if alpha is None else alpha
    _need(packed, "packed", torch.uint8, (N, K // 4))
    _need(alpha, "alpha", torch.float32)
    nbytes = L.bitnet_pack_workspace_bytes(N, K)
    ws = torch.empty((nbytes,), dtype=torch.uint8, device=dev) if ws is None else ws
    _native.check("bitnet_pack_ternary",
                  L.bitnet_pack_ternary(_ptr(W), N, K, eps, _ptr(packed), _ptr(alpha), _ptr(ws), ws.numel(),
                                        _stream(stream)))
    return packed, alpha


def _xdt(X: torch.Tensor) -> int:
    if X.dtype == torch.float32:
        return _native.F32
    if X.dtype == torch.bfloat16:
        return _native.BF16
    raise ValueError(f"X must be float32 or bfloat16, got {X.dtype}")


def bitnet_act_quant(X: torch.Tensor, gain=None, eps: float = 1e-5, fwht: bool = True, mode="int8",
                     codes=None, scale_x=None, stream=None):
    """RMSNorm -> optional FWHT -> per-token int8/int4 codes.  Returns (codes int8 [M,K], scale fp32 [M])."""
    L = _native.load()
    _need(X, "X")
    M, K = X.shape
    codes = torch.empty((M, K), dtype=torch.int8, device=X.device) if codes is None else codes
    scale_x = torch.empty((M,), dtype=torch.float32, device=X.device) if scale_x is None else scale_x
    _need(codes, "codes", torch.int8, (M, K))
    _need(scale_x, "scale_x", torch.float32, (M,))
    if gain is not None:
        _need(gain, "gain", torch.float32, (K,))
    _native.check("bitnet_act_quant",
                  L.bitnet_act_quant(_ptr(X), _xdt(X), M, K, _ptr(gain), eps, int(bool(fwht)), mode_id(mode),
                                     _ptr(codes), _ptr(scale_x), _stream(stream)))
    return codes, scale_x


def _need_pair(gate: torch.Tensor, up: torch.Tensor) -> None:
    _need(gate, "gate")
    _need(up, "up", gate.dtype, tuple(gate.shape))


def bitnet_act_quant_swiglu(gate: torch.Tensor, up: torch.Tensor, gain=None, eps: float = 1e-5, fwht: bool = True,
                            mode="int4", codes=None, scale_x=None, stream=None):
    """bitnet_act_quant on the SwiGLU product silu(gate) * up (formed in registers, never stored).
    Returns (codes int8 [M,K], scale fp32 [M])."""
    L = _native.load()
    _need_pair(gate, up)
    M, K = gate.shape
    codes = torch.empty((M, K), dtype=torch.int8, device=gate.device) if codes is None else codes
    scale_x = torch.empty((M,), dtype=torch.float32, device=gate.device) if scale_x is None else scale_x
    _need(codes, "codes", torch.int8, (M, K))
    _need(scale_x, "scale_x", torch.float32, (M,))
    if gain is not None:
        _need(gain, "gain", torch.float32, (K,))
    _native.check("bitnet_act_quant_swiglu",
                  L.bitnet_act_quant_swiglu(_ptr(gate), _ptr(up), _xdt(gate), M, K, _ptr(gain), eps, int(bool(fwht)),
                                            mode_id(mode), _ptr(codes), _ptr(scale_x), _stream(stream)))
    return codes, scale_x


def bitnet_hbitlinear_forward_swiglu(gate: torch.Tensor, up: torch.Tensor, packed: torch.Tensor, alpha: torch.Tensor,
                                     N: int, gain=None, eps: float = 1e-5, fwht: bool = True, mode="int4", out=None,
                                     ws=None, stream=None):
    """The H-BitLinear down projection of a BitNet v2 FFN on silu(gate) * up.  Returns out fp32 [M, N]."""
    L = _native.load()
    _need_pair(gate, up)
    M, K = gate.shape
    _need(packed, "packed", torch.uint8, (N, K // 4))
    _need(alpha, "alpha", torch.float32)
    if gain is not None:
        _need(gain, "gain", torch.float32, (K,))
    out = torch.empty((M, N), dtype=torch.float32, device=gate.device) if out is None else out
    _need(out, "out", torch.float32, (M, N))
    nbytes = L.bitnet_forward_workspace_bytes(M, K)
    ws = torch.empty((max(nbytes, 256),), dtype=torch.uint8, device=gate.device) if ws is None else ws
    _need(ws, "ws", torch.uint8)
    _native.check("bitnet_hbitlinear_forward_swiglu",
                  L.bitnet_hbitlinear_forward_swiglu(_ptr(gate), _ptr(up), _xdt(gate), M, K, _ptr(gain), eps,
                                                     int(bool(fwht)), mode_id(mode), _ptr(packed), _ptr(alpha), N,
                                                     _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def bitnet_kv_quant(kv: torch.Tensor, bits: int = 4, eps: float = 1e-5, dequant: bool = False, codes=None,
                    step=None, deq=None, stream=None):
    """Low-bit KV cache of a [..., S, D] key or value tensor (token 0 kept at int8).
    Returns (codes int8 [..., S, D], step fp32 [..., S], deq fp32 [..., S, D] or None)."""
    L = _native.load()
    _need(kv, "kv")
    S, D = kv.shape[-2], kv.shape[-1]
    BH = kv.numel() // (S * D) if S * D else 0
    codes = torch.empty(kv.shape, dtype=torch.int8, device=kv.device) if codes is None else codes
    step = torch.empty(kv.shape[:-1], dtype=torch.float32, device=kv.device) if step is None else step
    if dequant and deq is None:
        deq = torch.empty(kv.shape, dtype=torch.float32, device=kv.device)
    _need(codes, "codes", torch.int8, tuple(kv.shape))
    _need(step, "step", torch.float32, tuple(kv.shape[:-1]))
    if deq is not None:
        _need(deq, "deq", torch.float32, tuple(kv.shape))
    _native.check("bitnet_kv_quant", L.bitnet_kv_quant(_ptr(kv), _xdt(kv), BH, S, D, bits, eps, _ptr(codes),
                                                       _ptr(step), _ptr(deq), _stream(stream)))
    return codes, step, deq


def bitnet_ternary_gemm(codes: torch.Tensor, scale_x: torch.Tensor, mode, packed: torch.Tensor,
                        alpha: torch.Tensor, N: int, out=None, acc_out=None, ws=None, stream=None):
    """acc = codes @ t^T (exact int32) and out = acc * (alpha * scale_x / Q).  Returns out fp32 [M, N].

    ws (optional, uint8, >= bitnet_gemm_workspace_bytes) lets a problem with few output
    tiles split K; without it K is never split.  The result is the same either way."""
    L = _native.load()
    _need(codes, "codes", torch.int8)
    M, K = codes.shape
    _need(scale_x, "scale_x", torch.float32, (M,))
    _need(packed, "packed", torch.uint8, (N, K // 4))
    _need(alpha, "alpha", torch.float32)
    out = torch.empty((M, N), dtype=torch.float32, device=codes.device) if out is None else out
    _need(out, "out", torch.float32, (M, N))
    if acc_out is not None:
        _need(acc_out, "acc_out", torch.int32, (M, N))
    if ws is not None:
        _need(ws, "ws", torch.uint8)
    _native.check("bitnet_ternary_gemm",
                  L.bitnet_ternary_gemm(_ptr(codes), _ptr(scale_x), mode_id(mode), _ptr(packed), _ptr(alpha), M, N,
                                        K, _ptr(out), _ptr(acc_out), _ptr(ws), 0 if ws is None else ws.numel(),
                                        _stream(stream)))
    return out


def bitnet_hbitlinear_forward(X: torch.Tensor, packed: torch.Tensor, alpha: torch.Tensor, N: int, gain=None,
                              eps: float = 1e-5, fwht: bool = True, mode="int8", out=None, ws=None, stream=None):
    """The whole H-BitLinear forward.  Returns out fp32 [M, N]."""
    L = _native.load()
    _need(X, "X")
    M, K = X.shape
    _need(packed, "packed", torch.uint8, (N, K // 4))
    _need(alpha, "alpha", torch.float32)
    if gain is not None:
        _need(gain, "gain", torch.float32, (K,))
    out = torch.empty((M, N), dtype=torch.float32, device=X.device) if out is None else out
    _need(out, "out", torch.float32, (M, N))
    nbytes = L.bitnet_forward_workspace_bytes(M, K)
    ws = torch.empty((max(nbytes, 256),), dtype=torch.uint8, device=X.device) if ws is None else ws
    _need(ws, "ws", torch.uint8)
    _native.check("bitnet_hbitlinear_forward",
                  L.bitnet_hbitlinear_forward(_ptr(X), _xdt(X), M, K, _ptr(gain), eps, int(bool(fwht)),
                                              mode_id(mode), _ptr(packed), _ptr(alpha), N, _ptr(out), _ptr(ws),
                                              ws.numel(), _stream(stream)))
    return out


def bitnet_hbitlinear_forward_noalloc(X: torch.Tensor, packed: torch.Tensor, alpha: torch.Tensor, N: int,
                                      gain=None, eps: float = 1e-5, fwht: bool = True, mode="int8", out=None,
                                      stream=None):
    """The forward without a caller workspace, for callers that cannot allocate device memory
    (the scratch is a fixed 4 MiB array inside the library; see include/bitnet.h)."""
    L = _native.load()
    _need(X, "X")
    M, K = X.shape
    _need(packed, "packed", torch.uint8, (N, K // 4))
    _need(alpha, "alpha", torch.float32)
    if gain is not None:
        _need(gain, "gain", torch.float32, (K,))
    if out is None:
        raise ValueError("out must be given: this entry point is for callers that cannot allocate")
    _need(out, "out", torch.float32, (M, N))
    _native.check("bitnet_hbitlinear_forward_noalloc",
                  L.bitnet_hbitlinear_forward_noalloc(_ptr(X), _xdt(X), M, K, _ptr(gain), eps, int(bool(fwht)),
                                                      mode_id(mode), _ptr(packed), _ptr(alpha), N, _ptr(out),
                                                      _stream(stream)))
    return out


_OUT_DT = {torch.float32: 0, torch.bfloat16: 1}  # bitnet_dtype_t


def _out_dt(dtype) -> int:
    if dtype not in _OUT_DT:
        raise ValueError(f"output dtype must be torch.float32 or torch.bfloat16, got {dtype}")
    return _OUT_DT[dtype]


def bitnet_ternary_gemm_ex(codes: torch.Tensor, scale_x: torch.Tensor, mode, packed: torch.Tensor,
                           alpha: torch.Tensor, N: int, out_dtype=torch.bfloat16, out=None, acc_out=None,
                           stream=None):
    """bitnet_ternary_gemm with the output stored as out_dtype (fp32, or bf16 rounded to nearest even)."""
    L = _native.load()
    _need(codes, "codes", torch.int8)
    M, K = codes.shape
    _need(scale_x, "scale_x", torch.float32, (M,))
    _need(packed, "packed", torch.uint8, (N, K // 4))
    _need(alpha, "alpha", torch.float32)
    dt = _out_dt(out_dtype)
    out = torch.empty((M, N), dtype=out_dtype, device=codes.device) if out is None else out
    _need(out, "out", out_dtype, (M, N))
    if acc_out is not None:
        _need(acc_out, "acc_out", torch.int32, (M, N))
    _native.check("bitnet_ternary_gemm_ex",
                  L.bitnet_ternary_gemm_ex(_ptr(codes), _ptr(scale_x), mode_id(mode), _ptr(packed), _ptr(alpha), M,
                                           N, K, _ptr(out), dt, _ptr(acc_out), _stream(stream)))
    return out


def bitnet_hbitlinear_forward_ex(X: torch.Tensor, packed: torch.Tensor, alpha: torch.Tensor, N: int, gain=None,
                                 eps: float = 1e-5, fwht: bool = True, mode="int8", out_dtype=torch.bfloat16,
                                 out=None, ws=None, stream=None):
    """bitnet_hbitlinear_forward with the output stored as out_dtype (fp32, or bf16 rounded to nearest even)."""
    L = _native.load()
    _need(X, "X")
    M, K = X.shape
    _need(packed, "packed", torch.uint8, (N, K // 4))
    _need(alpha, "alpha", torch.float32)
    if gain is not None:
        _need(gain, "gain", torch.float32, (K,))
    dt = _out_dt(out_dtype)
    out = torch.empty((M, N), dtype=out_dtype, device=X.device) if out is None else out
    _need(out, "out", out_dtype, (M, N))
    nbytes = L.bitnet_forward_workspace_bytes(M, K)
    ws = torch.empty((max(nbytes, 256),), dtype=torch.uint8, device=X.device) if ws is None else ws
    _need(ws, "ws", torch.uint8)
    _native.check("bitnet_hbitlinear_forward_ex",
                  L.bitnet_hbitlinear_forward_ex(_ptr(X), _xdt(X), M, K, _ptr(gain), eps, int(bool(fwht)),
                                                 mode_id(mode), _ptr(packed), _ptr(alpha), N, _ptr(out), dt,
                                                 _ptr(ws), ws.numel(), _stream(stream)))
    return out


def bitnet_tl2_bytes(N: int, K: int) -> int:
    """Bytes of an N x K weight matrix in the TL2 format (20 per 96 weights of a row)."""
    return _native.load().bitnet_tl2_bytes(N, K)


def bitnet_pack_tl2(packed: torch.Tensor, K: int, tl2=None, stream=None):
    """2-bit packed weights [N, K/4] -> the TL2 format (5 bits per 3 weights), exactly.
    Returns uint8 [N, 20 * ceil(K/96)]."""
    L = _native.load()
    _need(packed, "packed", torch.uint8)
    N = packed.shape[0]
    if packed.shape[1] * 4 != K:
        raise ValueError(f"packed must be [N, K/4] = [N, {K // 4}], got {tuple(packed.shape)}")
    rb = L.bitnet_tl2_bytes(1, K)
    tl2 = torch.empty((N, rb), dtype=torch.uint8, device=packed.device) if tl2 is None else tl2
    _need(tl2, "tl2", torch.uint8, (N, rb))
    _native.check("bitnet_pack_tl2", L.bitnet_pack_tl2(_ptr(packed), N, K, _ptr(tl2), _stream(stream)))
    return tl2


def bitnet_ternary_gemm_tl2(codes: torch.Tensor, scale_x: torch.Tensor, mode, tl2: torch.Tensor,
                            alpha: torch.Tensor, N: int, out=None, acc_out=None, stream=None):
    """bitnet_ternary_gemm with TL2 weights (M <= 16).  Returns out fp32 [M, N]."""
    L = _native.load()
    _need(codes, "codes", torch.int8)
    M, K = codes.shape
    _need(scale_x, "scale_x", torch.float32, (M,))
    _need(tl2, "tl2", torch.uint8, (N, L.bitnet_tl2_bytes(1, K)))
    _need(alpha, "alpha", torch.float32)
    out = torch.empty((M, N), dtype=torch.float32, device=codes.device) if out is None else out
    _need(out, "out", torch.float32, (M, N))
    if acc_out is not None:
        _need(acc_out, "acc_out", torch.int32, (M, N))
    _native.check("bitnet_ternary_gemm_tl2",
                  L.bitnet_ternary_gemm_tl2(_ptr(codes), _ptr(scale_x), mode_id(mode), _ptr(tl2), _ptr(alpha), M, N,
                                            K, _ptr(out), _ptr(acc_out), _stream(stream)))
    return out


def bitnet_hbitlinear_forward_tl2(X: torch.Tensor, tl2: torch.Tensor, alpha: torch.Tensor, N: int, gain=None,
                                  eps: float = 1e-5, fwht: bool = True, mode="int8", out=None, ws=None,
                                  stream=None):
    """The whole H-BitLinear forward with TL2 weights (M <= 16).  Returns out fp32 [M, N]."""
    L = _native.load()
    _need(X, "X")
    M, K = X.shape
    _need(tl2, "tl2", torch.uint8, (N, L.bitnet_tl2_bytes(1, K)))
    _need(alpha, "alpha", torch.float32)
    if gain is not None:
        _need(gain, "gain", torch.float32, (K,))
    out = torch.empty((M, N), dtype=torch.float32, device=X.device) if out is None else out
    _need(out, "out", torch.float32, (M, N))
    nbytes = L.bitnet_forward_workspace_bytes(M, K)
    ws = torch.empty((max(nbytes, 256),), dtype=torch.uint8, device=X.device) if ws is None else ws
    _need(ws, "ws", torch.uint8)
    _native.check("bitnet_hbitlinear_forward_tl2",
                  L.bitnet_hbitlinear_forward_tl2(_ptr(X), _xdt(X), M, K, _ptr(gain), eps, int(bool(fwht)),
                                                  mode_id(mode), _ptr(tl2), _ptr(alpha), N, _ptr(out), _ptr(ws),
                                                  ws.numel(), _stream(stream)))
    return out


class KV4Cache:
    """The 4-bit paged KV cache: six tensors on one CUDA device (layout in include/bitnet.h).

    k_codes, v_codes uint8 [pages, heads, page_size, dim/2]; k_step, v_step fp32 [pages, heads, page_size];
    k_bos, v_bos int8 [pages, heads, dim].  KV4Cache.empty allocates them (page 16, 32, 64, 128 or 256;
    dim 64, 128 or 256).  The object keeps the tensors' addresses; a batch of sequences is described to the
    calls by three int32 CUDA tensors:

        block_table [B, max_pages]  page of position s of sequence b: block_table[b, s // page_size]; may be a part
                                    of the columns of a wider table
        kv_lens     [B]             positions in the cache, this step's rows included
        q_starts    [B + 1]         sequence b owns rows q_starts[b]:q_starts[b + 1] of the token tensors, at
                                    its last positions

    A step of a model writes its new keys and values, then attends:

        bitnet_kv4_write(k, v, cache, block_table, kv_lens, q_starts)
        out = bitnet_kv4_attention(q, cache, block_table, kv_lens, q_starts)
    """

    def __init__(self, k_codes, v_codes, k_step, v_step, k_bos, v_bos):
        _need(k_codes, "k_codes", torch.uint8)
        if k_codes.dim() != 4:
            raise ValueError(f"k_codes must be [pages, heads, page_size, dim/2], got {tuple(k_codes.shape)}")
        pages, heads, page, half = k_codes.shape
        self.device = k_codes.device
        self.pages, self.heads, self.page_size, self.dim = pages, heads, page, 2 * half
        for name, t, dtype, shape in (("v_codes", v_codes, torch.uint8, (pages, heads, page, half)),
                                      ("k_step", k_step, torch.float32, (pages, heads, page)),
                                      ("v_step", v_step, torch.float32, (pages, heads, page)),
                                      ("k_bos", k_bos, torch.int8, (pages, heads, self.dim)),
                                      ("v_bos", v_bos, torch.int8, (pages, heads, self.dim))):
            _need(t, name, dtype, shape)
            if t.device != self.device:
                raise ValueError(f"{name} must be on {self.device}, got {t.device}")
        self.k_codes, self.v_codes, self.k_step, self.v_step = k_codes, v_codes, k_step, v_step
        self.k_bos, self.v_bos = k_bos, v_bos
        self._c = _native.Kv4Cache(k_codes.data_ptr(), v_codes.data_ptr(), k_step.data_ptr(), v_step.data_ptr(),
                                   k_bos.data_ptr(), v_bos.data_ptr(), pages, heads, page, self.dim)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, pages: int, heads: int, dim: int, page_size: int = 64, device="cuda") -> "KV4Cache":
        """A cache whose memory is not initialised (rows that no write has reached are never read)."""
        if dim % 2:
            raise ValueError(f"dim must be even, got {dim}")
        codes = [torch.empty((pages, heads, page_size, dim // 2), dtype=torch.uint8, device=device) for _ in range(2)]
        steps = [torch.empty((pages, heads, page_size), dtype=torch.float32, device=device) for _ in range(2)]
        bos = [torch.empty((pages, heads, dim), dtype=torch.int8, device=device) for _ in range(2)]
        return cls(*codes, *steps, *bos)


def _kv4_batch(cache: KV4Cache, block_table: torch.Tensor, kv_lens: torch.Tensor, q_starts: torch.Tensor):
    if not isinstance(cache, KV4Cache):
        raise TypeError("cache must be a KV4Cache")
    dev = cache.device
    try:  # a step of a model makes these calls for each layer: one expression first, the reasons after it
        B, width = block_table.shape
        good = (kv_lens.shape == (B,) and q_starts.shape == (B + 1,) and
                block_table.dtype is torch.int32 and kv_lens.dtype is torch.int32 and q_starts.dtype is torch.int32 and
                block_table.device == dev and kv_lens.device == dev and q_starts.device == dev and
                kv_lens.is_contiguous() and q_starts.is_contiguous())
        stride, unit = block_table.stride()
        good = good and (block_table.is_contiguous() or ((unit == 1 or width == 1) and (stride >= width or B == 1)))
    except (AttributeError, ValueError):
        good = False
    if not good:
        B = kv_lens.shape[0] if isinstance(kv_lens, torch.Tensor) and kv_lens.dim() == 1 else -1
        _need(kv_lens, "kv_lens", torch.int32, (B,))
        _need(q_starts, "q_starts", torch.int32, (B + 1,))
        _need(block_table[:0] if isinstance(block_table, torch.Tensor) and block_table.dim() else block_table, "block_table", torch.int32)
        if block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError(f"block_table must be [{B}, max_pages], got {tuple(block_table.shape)}")
        if block_table.numel() and (block_table.stride(1) != 1 or block_table.stride(0) < block_table.shape[1]):
            raise ValueError("block_table's rows must be contiguous and lie one behind the other")
        raise ValueError(f"block_table, kv_lens and q_starts must be on the cache's device {dev}")
    return _native.Kv4Batch(block_table.data_ptr(), kv_lens.data_ptr(), q_starts.data_ptr(), max(stride, width), B, width)


def _rows(t: torch.Tensor, name: str, cache: KV4Cache, heads=None):
    """Checks a [T, heads, dim] tensor whose rows of dim lie anywhere; returns (T, token stride, head stride)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != cache.device:
        raise ValueError(f"{name} must be a CUDA tensor on the cache's device {cache.device}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[2] != cache.dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must have shape [T, {'heads' if heads is None else heads}, {cache.dim}], "
                         f"got {tuple(shape)}")
    if stride[2] != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    # the stride of a dimension of one says nothing
    return shape[0], stride[0] if shape[0] > 1 else 0, stride[1] if shape[1] > 1 else 0


def _empty(like: torch.Tensor, shape, stream, dtype=None) -> torch.Tensor:
    """Memory for a call on `stream`, of the type (unless given) and device of `like`, from that stream's pool: no other
    stream's work still uses it, or will before the call is done with it."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype) if dtype else like.new_empty(*shape)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype or like.dtype)


def _kv4_call(cache: KV4Cache, fn: str, stream, *args) -> None:
    """The call with the cache's device current (a kernel is launched on the current one), on its current stream."""
    index = cache.device.index
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if index == torch.cuda.current_device():
        status = getattr(_native.load(), fn)(*args, handle)
    else:
        with torch.cuda.device(index):
            status = getattr(_native.load(), fn)(*args, handle)
    if status:
        _native.check(fn, status)


def bitnet_kv4_write(k: torch.Tensor, v: torch.Tensor, cache: KV4Cache, block_table: torch.Tensor,
                     kv_lens: torch.Tensor, q_starts: torch.Tensor, bits: int = 4, eps: float = 1e-5,
                     stream=None) -> None:
    """Quantise the new rows k, v [T, heads, dim] (fp32 or bf16, any token and head strides) into the cache, at
    the last positions of their sequences.  Position 0 is kept at 8 bits, the others at `bits` (4: absmean,
    3: absmax).  kv_lens counts the new rows."""
    batch = _kv4_batch(cache, block_table, kv_lens, q_starts)
    T, kts, khs = _rows(k, "k", cache, cache.heads)
    Tv, vts, vhs = _rows(v, "v", cache, cache.heads)
    if Tv != T or v.dtype != k.dtype:
        raise ValueError(f"v must have {T} rows of {k.dtype}, got {Tv} of {v.dtype}")
    _kv4_call(cache, "bitnet_kv4_write", stream, k.data_ptr(), v.data_ptr(), _xdt(k), T, kts, khs, vts, vhs,
              cache._ref, ctypes.byref(batch), bits, eps)


def bitnet_kv4_read(cache: KV4Cache, block_table: torch.Tensor, kv_lens: torch.Tensor, q_starts: torch.Tensor,
                    total: int, dtype=torch.float32, k_out=None, v_out=None, stream=None):
    """The cached values of the batch's rows (the last q_starts[b+1] - q_starts[b] positions of sequence b) as
    (k, v), each [total, heads, dim] of dtype.  Rows that belong to no sequence are left as they are."""
    batch = _kv4_batch(cache, block_table, kv_lens, q_starts)
    dt = _out_dt(dtype)
    shape = (total, cache.heads, cache.dim)
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is not None:
            _need(t, name, dtype, shape)
            if t.device != cache.device:
                raise ValueError(f"{name} must be on the cache's device {cache.device}")
    k_out = _empty(cache.k_step, shape, stream, dtype) if k_out is None else k_out
    v_out = _empty(cache.k_step, shape, stream, dtype) if v_out is None else v_out
    _kv4_call(cache, "bitnet_kv4_read", stream, cache._ref, ctypes.byref(batch), total, k_out.data_ptr(),
              v_out.data_ptr(), dt)
    return k_out, v_out


@functools.lru_cache(maxsize=4096)
def _kv4_workspace_bytes(index: int, *sizes: int) -> int:
    """The size on CUDA device `index` (it depends on the number of SMs), which is asked for with that device current."""
    with torch.cuda.device(index):
        return _native.load().bitnet_kv4_attention_workspace_bytes(*sizes)


def bitnet_kv4_attention_workspace_bytes(T: int, q_heads: int, heads: int, dim: int, batch: int, device=None) -> int:
    """Workspace of bitnet_kv4_attention for T rows of q_heads over a cache of `heads` key heads (0: sizes it refuses), on
    `device` (the current one unless given).  A smaller T can need more, as few rows are divided among more CTAs."""
    if not torch.cuda.is_available():
        return _native.load().bitnet_kv4_attention_workspace_bytes(T, q_heads, heads, dim, batch)
    index = None if device is None else device if isinstance(device, int) else torch.device(device).index
    return _kv4_workspace_bytes(torch.cuda.current_device() if index is None else index, T, q_heads, heads, dim, batch)


def bitnet_kv4_attention(q: torch.Tensor, cache: KV4Cache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                         q_starts: torch.Tensor, scale=None, causal: bool = True, window: int = 0, max_q: int = 0,
                         return_lse: bool = False, out=None, lse=None, ws=None, stream=None):
    """Softmax attention of q [T, q_heads, dim] (fp32 or bf16, any token and head strides) over the cached keys and
    values of each row's sequence; query head h reads key head h // (q_heads // heads).  scale defaults to
    dim ** -0.5; window > 0 limits a causal row to its last `window` positions; max_q, the largest number
    of rows of a sequence, is a hint for the choice of kernel (worth giving where q has many rows of nobody).
    Rows that see nothing give zeros (lse -inf).

    Returns out [T, q_heads, dim] of q's dtype, or (out, lse fp32 [T, q_heads]) with return_lse.  Calls that may
    run at the same time need workspaces of their own."""
    batch = _kv4_batch(cache, block_table, kv_lens, q_starts)
    T, qts, qhs = _rows(q, "q", cache)
    dt, heads, dev = _xdt(q), q.shape[1], cache.device
    if out is None:
        out = _empty(q, (T, heads, cache.dim), stream)
    else:
        _need(out, "out", q.dtype, (T, heads, cache.dim))
    if lse is None:
        lse = _empty(cache.k_step, (T, heads), stream) if return_lse else None
    else:
        _need(lse, "lse", torch.float32, (T, heads))
    if ws is None:
        ws = _empty(cache.k_codes,
                    (_kv4_workspace_bytes(dev.index, T, heads, cache.heads, cache.dim, batch.batch) or 256,), stream)
    else:
        _need(ws, "ws", torch.uint8)
    if out.device != dev or ws.device != dev or (lse is not None and lse.device != dev):
        raise ValueError(f"out, lse and ws must be on the cache's device {dev}")
    scale = cache.dim ** -0.5 if scale is None else scale
    _kv4_call(cache, "bitnet_kv4_attention", stream, q.data_ptr(), dt, T, heads, qts, qhs, cache._ref,
              ctypes.byref(batch), scale, int(bool(causal)), window, max_q, out.data_ptr(),
              None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.numel())
    return (out, lse) if return_lse else out


def bitnet_get_last_device_status(stream=None) -> int:
    """Synchronise the stream, return and clear the kernels' timeout status word."""
    return _native.load().bitnet_get_last_device_status(_stream(stream))


def bitnet_selftest_wait_timeout(limit_us: int, stream=None) -> None:
    _native.check("bitnet_selftest_wait_timeout",
                  _native.load().bitnet_selftest_wait_timeout(limit_us, _stream(stream)))


class HBitLinear:
    """Pack once, forward many: an H-BitLinear layer over a fixed weight matrix.

    W is [out_features, in_features] fp32 on a CUDA device.  fwht=True gives the
    H-BitLinear of the BitNet v2 page (Wo / Wdown); fwht=False the plain BitLinear.
    The layer keeps one forward workspace and reuses it, so calls of the same layer
    on different streams must be ordered (events, or one stream)."""

    def __init__(self, W: torch.Tensor, mode="int8", fwht: bool = True, eps: float = 1e-5, gain=None):
        self.N, self.K = W.shape
        self.mode = mode_id(mode)
        self.fwht = bool(fwht)
        self.eps = float(eps)
        self.gain = gain
        self.packed, self.alpha = bitnet_pack_ternary(W, eps)
        self._ws = None

    def workspace(self, M: int, device) -> torch.Tensor:
        need = max(bitnet_forward_workspace_bytes(M, self.K), 256)
        if self._ws is None or self._ws.numel() < need or self._ws.device != device:
            self._ws = torch.empty((need,), dtype=torch.uint8, device=device)
        return self._ws

    def __call__(self, X: torch.Tensor, out=None, stream=None) -> torch.Tensor:
        return bitnet_hbitlinear_forward(X, self.packed, self.alpha, self.N, gain=self.gain, eps=self.eps,
                                         fwht=self.fwht, mode=self.mode, out=out,
                                         ws=self.workspace(X.shape[0], X.device), stream=stream)
