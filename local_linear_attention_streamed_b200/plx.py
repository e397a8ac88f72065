"""Thin ctypes binding over libplx.so (include/plx.h).

Argument marshalling only: torch tensors are passed as raw device pointers and
the current torch stream; every step of the computation runs in the library's
CUDA kernels.  Loading fails loudly when the library is missing; there is no
fallback.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

import torch

PLX_F32 = 0
PLX_BF16 = 1
PLX_ERR_CUDA = -4

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libplx.so")

# Exported symbols and their C signatures (mirrors include/plx.h).
_vp, _i, _sz, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
SIGNATURES = {
    "plx_prefill": (_i, [_vp] * 5 + [_i] * 5),
    "plx_prefill_ex": (_i, [_vp] * 5 + [_i] * 6 + [_vp]),
    "plx_decode": (_i, [_vp] * 6 + [_i] * 4),
    "plx_decode_ex": (_i, [_vp] * 6 + [_i] * 5 + [_vp, _sz, _vp]),
    "plx_decode_workspace_bytes": (_sz, [_i] * 4),
    "plx_decode_num_splits": (_i, [_i] * 4),
    "plx_decode_uses_tc": (_i, [_i] * 4),
    "plx_decode_noalloc": (_i, [_vp] * 6 + [_i] * 4 + [_vp]),
    "plx_decode_gqa": (_i, [_vp] * 6 + [_i] * 5 + [_vp, _sz, _vp]),
    "plx_decode_gqa_workspace_bytes": (_sz, [_i] * 5),
    "plx_qkr_norm_rope": (_i, [_vp, _vp] + [_i] * 4 + [_f, _f, _vp]),
    "plx_layer_workspace_bytes": (_sz, [_i] * 4),
    "plx_layer_forward": (_i, [_vp] * 7 + [_i] * 4 + [_vp, _sz, _vp]),
    "plx_layer_fp8_workspace_bytes": (_sz, [_i] * 4),
    "plx_layer_forward_fp8": (_i, [_vp] * 7 + [_i] * 4 + [_vp, _sz, _vp]),
    "plx_prefill_window": (_i, [_vp] * 5 + [_i] * 6 + [_vp]),
    "plx_prefill_block_sparse": (_i, [_vp] * 5 + [_i] * 4 + [_vp, _vp]),
    "plx_prefill_gqa": (_i, [_vp] * 5 + [_i] * 6 + [_vp]),
    "plx_decode_window": (_i, [_vp] * 6 + [_i] * 7 + [_vp, _sz, _vp]),
    "plx_decode_window_workspace_bytes": (_sz, [_i] * 6),
    "plx_prefill_train": (_i, [_vp] * 8 + [_i] * 5 + [_vp]),
    "plx_prefill_bwd_workspace_bytes": (_sz, [_i] * 4),
    "plx_prefill_bwd": (_i, [_vp] * 13 + [_i] * 5 + [_vp, _sz, _vp]),
    "plx_prefill_train_window": (_i, [_vp] * 8 + [_i] * 5 + [_vp]),
    "plx_prefill_bwd_window": (_i, [_vp] * 13 + [_i] * 5 + [_vp, _sz, _vp]),
    "plx_prefill_train_gqa": (_i, [_vp] * 8 + [_i] * 6 + [_vp]),
    "plx_prefill_train_ex": (_i, [_vp] * 8 + [_i] * 7 + [_vp]),
    "plx_prefill_bwd_ex": (_i, [_vp] * 13 + [_i] * 7 + [_vp, _sz, _vp]),
    "plx_prefill_gqa_window": (_i, [_vp] * 5 + [_i] * 6 + [_vp]),
    "plx_prefill_bwd_gqa": (_i, [_vp] * 13 + [_i] * 6 + [_vp, _sz, _vp]),
    "plx_prefill_dilated": (_i, [_vp] * 5 + [_i] * 7 + [_vp]),
    "plx_kv_quantize_fp8": (_i, [_vp, _vp, _vp, ctypes.c_longlong, _i, _vp]),
    "plx_decode_fp8kv_workspace_bytes": (_sz, [_i] * 5),
    "plx_decode_fp8kv": (_i, [_vp] * 8 + [_i] * 5 + [_vp, _sz, _vp]),
    "plx_kv_quantize_int4": (_i, [_vp] * 3 + [ctypes.c_longlong, _i, _vp]),
    "plx_kv_dequantize_int4": (_i, [_vp] * 3 + [ctypes.c_longlong, _i, _vp]),
    "plx_kv_append_int4": (_i, [_vp] * 9 + [_i] * 4 + [_vp]),
    "plx_decode_int4kv_workspace_bytes": (_sz, [_i] * 5),
    "plx_decode_int4kv": (_i, [_vp] * 8 + [_i] * 5 + [_vp, _sz, _vp]),
    "plx_decode_weights_workspace_bytes": (_sz, [_i] * 5),
    "plx_decode_weights": (_i, [_vp] * 8 + [_i] * 5 + [_vp, _sz, _vp]),
    "plx_decode_int4kv_weights": (_i, [_vp] * 10 + [_i] * 5 + [_vp, _sz, _vp]),
    "plx_cache_evict": (_i, [_i] + [_vp] * 8 + [_i] * 7 + [_vp]),
    "plx_get_device_status": (_i, [_vp]),
    "plx_status_string": (ctypes.c_char_p, [_i]),
    "plx_last_cuda_error": (ctypes.c_char_p, []),
    "plx_abi_version": (_i, []),
}


class PlxError(RuntimeError):
    def __init__(self, code: int, where: str):
        msg = f"{where}: {status_string(code)} (code {code})"
        if code == PLX_ERR_CUDA:
            msg += f": {lib.plx_last_cuda_error().decode()}"
        super().__init__(msg)
        self.code = code


def _load():
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                           "(python -m local_linear_attention_streamed_b200._build)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def status_string(code: int) -> str:
    return lib.plx_status_string(int(code)).decode()


def _check(rc: int, where: str) -> None:
    if rc != 0:
        raise PlxError(rc, where)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return PLX_BF16
    if t.dtype == torch.float32:
        return PLX_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _dev(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def prefill(Q, K, V, R, causal: bool = True, out=None, stream=None):
    """Parallax prefill over [B, H, N, d] tensors (bf16 or fp32); returns out."""
    B, H, N, d = Q.shape
    for n, t in (("K", K), ("V", V), ("R", R)):
        if t.shape != Q.shape or t.dtype != Q.dtype:
            raise ValueError(f"{n} must match Q in shape and dtype")
    if out is None:
        out = torch.empty_like(Q)
    rc = lib.plx_prefill_ex(_dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(R, "R"), _dev(out, "out"),
                            B, H, N, d, int(bool(causal)), _dtype_code(Q), _stream_ptr(stream))
    _check(rc, "plx_prefill_ex")
    return out


def prefill_window(Q, K, V, R, window: int, out=None, stream=None):
    """Sliding-window causal prefill (query i sees its last `window` keys); returns out."""
    B, H, N, d = Q.shape
    for n, t in (("K", K), ("V", V), ("R", R)):
        if t.shape != Q.shape or t.dtype != Q.dtype:
            raise ValueError(f"{n} must match Q in shape and dtype")
    if out is None:
        out = torch.empty_like(Q)
    rc = lib.plx_prefill_window(_dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(R, "R"), _dev(out, "out"),
                                B, H, N, d, int(window), _dtype_code(Q), _stream_ptr(stream))
    _check(rc, "plx_prefill_window")
    return out


def prefill_gqa(Q, K, V, R, causal: bool = True, out=None, stream=None, window=None):
    """bf16 prefill with grouped KV heads: Q, R [B, H, N, d]; K, V [B, Hkv, N, d]
    (``window``: the last W keys of each query, as prefill_window)."""
    B, H, N, d = Q.shape
    Hkv = K.shape[1]
    if K.shape != (B, Hkv, N, d) or V.shape != K.shape or R.shape != Q.shape:
        raise ValueError("K, V must be [B, Hkv, N, d] and R like Q")
    if out is None:
        out = torch.empty_like(Q)
    if window is None:
        rc = lib.plx_prefill_gqa(_dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(R, "R"), _dev(out, "out"),
                                 B, H, Hkv, N, d, int(bool(causal)), _stream_ptr(stream))
        _check(rc, "plx_prefill_gqa")
    else:
        rc = lib.plx_prefill_gqa_window(_dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(R, "R"), _dev(out, "out"),
                                        B, H, Hkv, N, d, int(window), _stream_ptr(stream))
        _check(rc, "plx_prefill_gqa_window")
    return out


def prefill_block_sparse(Q, K, V, R, block_mask, out=None, stream=None):
    """Block-sparse causal prefill: ``block_mask`` is a host array [ceil(N/128), ceil(N/64)]
    (truthy = the 64-key block is visible to the 128-query tile); returns out."""
    import numpy as np
    B, H, N, d = Q.shape
    for n, t in (("K", K), ("V", V), ("R", R)):
        if t.shape != Q.shape or t.dtype != Q.dtype:
            raise ValueError(f"{n} must match Q in shape and dtype")
    m = np.ascontiguousarray(np.asarray(block_mask).astype(np.uint8))
    if m.shape != ((N + 127) // 128, (N + 63) // 64):
        raise ValueError("block_mask must be [ceil(N/128), ceil(N/64)]")
    if out is None:
        out = torch.empty_like(Q)
    rc = lib.plx_prefill_block_sparse(_dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(R, "R"), _dev(out, "out"),
                                      B, H, N, d, m.ctypes.data, _stream_ptr(stream))
    _check(rc, "plx_prefill_block_sparse")
    return out


def decode_window(q, r, Kcache, Vcache, seqlens, window: int, out=None, workspace=None, stream=None):
    """Sliding-window decode step: each query sees the last `window` keys of its sequence.

    Kcache/Vcache are [B, Hkv, L, d] with H a multiple of Hkv (Hkv == H: one KV head per head).
    """
    B, H, d = q.shape
    Hkv, L = Kcache.shape[1], Kcache.shape[2]
    if out is None:
        out = torch.empty_like(q)
    ws, wsb = (0, 0) if workspace is None else (_dev(workspace, "workspace"),
                                                workspace.numel() * workspace.element_size())
    rc = lib.plx_decode_window(_dev(q, "q"), _dev(r, "r"), _dev(Kcache, "Kcache"), _dev(Vcache, "Vcache"),
                               _dev(seqlens, "seqlens"), _dev(out, "out"), B, H, Hkv, L, d, int(window),
                               _dtype_code(q), ws, wsb, _stream_ptr(stream))
    _check(rc, "plx_decode_window")
    return out


def _kv_heads(Q, K, V):
    """KV heads of K and V ([B, Hkv, N, d], H a multiple of Hkv)."""
    B, H, N, d = Q.shape
    Hkv = K.shape[1]
    if K.shape != (B, Hkv, N, d) or V.shape != K.shape or Hkv < 1 or H % Hkv:
        raise ValueError("K, V must be [B, Hkv, N, d] with H a multiple of Hkv")
    return Hkv


def prefill_train(Q, K, V, R, causal: bool = True, stream=None, window=None):
    """bf16 prefill that also saves the backward pass's inputs (``window``:
    the sliding-window prefill of prefill_window).  K and V may have fewer
    heads than Q (grouped KV heads, as prefill_gqa).

    Returns (out, vbar, lse, tbar): out bf16 [B, H, N, d], vbar fp32
    [B, H, N, d], lse and tbar fp32 [B, H, N] (see plx_prefill_train in
    include/plx.h).
    """
    B, H, N, d = Q.shape
    Hkv = _kv_heads(Q, K, V)
    for n, t in (("K", K), ("V", V), ("R", R)):
        if t.dtype != Q.dtype:
            raise ValueError(f"{n} must match Q's dtype")
    if R.shape != Q.shape:
        raise ValueError("R must match Q's shape")
    if Q.dtype != torch.bfloat16:
        raise TypeError("prefill_train takes bf16 tensors")
    out = torch.empty_like(Q)
    vbar = torch.empty(Q.shape, dtype=torch.float32, device=Q.device)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=Q.device)
    tbar = torch.empty((B, H, N), dtype=torch.float32, device=Q.device)
    if Hkv != H:
        rc = lib.plx_prefill_train_ex(_dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(R, "R"), _dev(out, "out"),
                                      _dev(vbar, "vbar"), _dev(lse, "lse"), _dev(tbar, "tbar"), B, H, Hkv, N, d,
                                      int(bool(causal)), 0 if window is None else int(window), _stream_ptr(stream))
        _check(rc, "plx_prefill_train_ex")
    elif window is None:
        rc = lib.plx_prefill_train(_dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(R, "R"), _dev(out, "out"),
                                   _dev(vbar, "vbar"), _dev(lse, "lse"), _dev(tbar, "tbar"), B, H, N, d,
                                   int(bool(causal)), _stream_ptr(stream))
        _check(rc, "plx_prefill_train")
    else:
        rc = lib.plx_prefill_train_window(_dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(R, "R"),
                                          _dev(out, "out"), _dev(vbar, "vbar"), _dev(lse, "lse"),
                                          _dev(tbar, "tbar"), B, H, N, d, int(window), _stream_ptr(stream))
        _check(rc, "plx_prefill_train_window")
    return out, vbar, lse, tbar


def prefill_bwd_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(lib.plx_prefill_bwd_workspace_bytes(B, H, N, d))


def prefill_backward(Q, K, V, R, out, vbar, lse, tbar, dO, causal: bool = True, grads=None,
                     workspace=None, stream=None, window=None):
    """Gradients (dQ, dK, dV, dR) of sum(out * dO) for one bf16 prefill.

    ``out, vbar, lse, tbar`` are what prefill_train returned for the same
    inputs; ``grads`` optionally gives the four output tensors.  With grouped
    KV heads (K, V [B, Hkv, N, d]) dK and dV have K's shape: each sums over
    its group's query heads.
    """
    B, H, N, d = Q.shape
    Hkv = _kv_heads(Q, K, V)
    for n, t in (("K", K), ("V", V)):
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{n} must be bf16")
    for n, t in (("R", R), ("out", out), ("dO", dO)):
        if t.shape != Q.shape or t.dtype != torch.bfloat16:
            raise ValueError(f"{n} must be bf16 of Q's shape")
    if vbar.shape != Q.shape or vbar.dtype != torch.float32:
        raise ValueError("vbar must be fp32 of Q's shape")
    for n, t in (("lse", lse), ("tbar", tbar)):
        if t.shape != (B, H, N) or t.dtype != torch.float32:
            raise ValueError(f"{n} must be fp32 [B, H, N]")
    if grads is None:
        grads = (torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V), torch.empty_like(Q))
    dQ, dK, dV, dR = grads
    ws, wsb = (0, 0) if workspace is None else (_dev(workspace, "workspace"),
                                                workspace.numel() * workspace.element_size())
    args = (_dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(R, "R"), _dev(out, "out"), _dev(vbar, "vbar"),
            _dev(lse, "lse"), _dev(tbar, "tbar"), _dev(dO, "dO"), _dev(dQ, "dQ"), _dev(dK, "dK"),
            _dev(dV, "dV"), _dev(dR, "dR"), B, H, N, d)
    if Hkv != H:
        rc = lib.plx_prefill_bwd_ex(*args[:14], H, Hkv, N, d, int(bool(causal)), 0 if window is None else int(window),
                                    ws, wsb, _stream_ptr(stream))
        _check(rc, "plx_prefill_bwd_ex")
    elif window is None:
        rc = lib.plx_prefill_bwd(*args, int(bool(causal)), ws, wsb, _stream_ptr(stream))
        _check(rc, "plx_prefill_bwd")
    else:
        rc = lib.plx_prefill_bwd_window(*args, int(window), ws, wsb, _stream_ptr(stream))
        _check(rc, "plx_prefill_bwd_window")
    return dQ, dK, dV, dR


class ParallaxAttention(torch.autograd.Function):
    """Autograd wrapper: forward = prefill_train, backward = prefill_backward (bf16)."""

    @staticmethod
    def forward(ctx, Q, K, V, R, causal=True, window=None):
        Q, K, V, R = (t.contiguous() for t in (Q, K, V, R))
        out, vbar, lse, tbar = prefill_train(Q, K, V, R, causal, window=window)
        ctx.save_for_backward(Q, K, V, R, out, vbar, lse, tbar)
        ctx.causal = causal
        ctx.window = window
        return out

    @staticmethod
    def backward(ctx, dO):
        Q, K, V, R, out, vbar, lse, tbar = ctx.saved_tensors
        dQ, dK, dV, dR = prefill_backward(Q, K, V, R, out, vbar, lse, tbar,
                                          dO.contiguous().to(torch.bfloat16), ctx.causal, window=ctx.window)
        return dQ, dK, dV, dR, None, None


def parallax_attention(Q, K, V, R, causal: bool = True, window=None):
    """Differentiable bf16 Parallax attention over [B, H, N, d] (d in {64, 128});
    ``window`` (None or W >= 1) makes it the sliding-window prefill; K and V
    may have fewer heads (grouped KV heads, with or without a window)."""
    return ParallaxAttention.apply(Q, K, V, R, causal, window)


def decode_workspace_bytes(B: int, H: int, L: int, d: int) -> int:
    return int(lib.plx_decode_workspace_bytes(B, H, L, d))


def decode(q, r, Kcache, Vcache, seqlens, out=None, workspace=None, stream=None):
    """One decode step: q, r [B, H, d]; caches [B, H, L, d]; seqlens int32 [B]."""
    B, H, L, d = Kcache.shape
    if q.shape != (B, H, d) or r.shape != (B, H, d) or Vcache.shape != Kcache.shape:
        raise ValueError("shape mismatch")
    if seqlens.dtype != torch.int32 or seqlens.shape != (B,):
        raise ValueError("seqlens must be int32 [B]")
    if out is None:
        out = torch.empty_like(q)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()
    rc = lib.plx_decode_ex(_dev(q, "q"), _dev(r, "r"), _dev(Kcache, "Kcache"), _dev(Vcache, "Vcache"),
                           _dev(seqlens, "seqlens"), _dev(out, "out"), B, H, L, d, _dtype_code(q),
                           ws_ptr, ws_bytes, _stream_ptr(stream))
    _check(rc, "plx_decode_ex")
    return out


def decode_noalloc(q, r, Kcache, Vcache, seqlens, out=None, stream=None):
    """As decode() for bf16, through plx_decode_noalloc: no device memory is allocated
    (the library's fixed scratch array is used)."""
    B, H, L, d = Kcache.shape
    if q.shape != (B, H, d) or r.shape != (B, H, d) or Vcache.shape != Kcache.shape:
        raise ValueError("shape mismatch")
    if seqlens.dtype != torch.int32 or seqlens.shape != (B,):
        raise ValueError("seqlens must be int32 [B]")
    if out is None:
        out = torch.empty_like(q)
    rc = lib.plx_decode_noalloc(_dev(q, "q"), _dev(r, "r"), _dev(Kcache, "Kcache"),
                                _dev(Vcache, "Vcache"), _dev(seqlens, "seqlens"), _dev(out, "out"),
                                B, H, L, d, _stream_ptr(stream))
    _check(rc, "plx_decode_noalloc")
    return out


def decode_gqa(q, r, Kcache, Vcache, seqlens, out=None, workspace=None, stream=None):
    """One bf16 decode step with grouped KV heads: q, r [B, H, d]; caches [B, Hkv, L, d]
    (query head h reads KV head h // (H // Hkv)); seqlens int32 [B]."""
    B, Hkv, L, d = Kcache.shape
    H = q.shape[1]
    if q.shape != (B, H, d) or r.shape != (B, H, d) or Vcache.shape != Kcache.shape:
        raise ValueError("shape mismatch")
    if seqlens.dtype != torch.int32 or seqlens.shape != (B,):
        raise ValueError("seqlens must be int32 [B]")
    if out is None:
        out = torch.empty_like(q)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()
    rc = lib.plx_decode_gqa(_dev(q, "q"), _dev(r, "r"), _dev(Kcache, "Kcache"), _dev(Vcache, "Vcache"),
                            _dev(seqlens, "seqlens"), _dev(out, "out"), B, H, Hkv, L, d,
                            ws_ptr, ws_bytes, _stream_ptr(stream))
    _check(rc, "plx_decode_gqa")
    return out


def prefill_dilated(Q, K, V, R, dilation: int, window: int = 0, out=None, stream=None):
    """Dilated causal prefill: query i sees keys i, i - r, i - 2r, ... (the last
    ``window`` of them; all when 0).  Q, R [B, H, N, d]; K, V [B, Hkv, N, d]."""
    B, H, N, d = Q.shape
    Hkv = K.shape[1]
    if out is None:
        out = torch.empty_like(Q)
    rc = lib.plx_prefill_dilated(_dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(R, "R"), _dev(out, "out"),
                                 B, H, Hkv, N, d, dilation, window, _stream_ptr(stream))
    _check(rc, "plx_prefill_dilated")
    return out


def kv_quantize_fp8(X, codes=None, scales=None, stream=None):
    """Per-row dynamic e4m3 quantisation of bf16 cache rows X[..., d]:
    returns (codes uint8 [..., d], scales float32 [...])."""
    d = X.shape[-1]
    rows = X.numel() // d
    if codes is None:
        codes = torch.empty(X.shape, dtype=torch.uint8, device=X.device)
    if scales is None:
        scales = torch.empty(X.shape[:-1], dtype=torch.float32, device=X.device)
    rc = lib.plx_kv_quantize_fp8(_dev(X, "X"), _dev(codes, "codes"), _dev(scales, "scales"), rows, d,
                                 _stream_ptr(stream))
    _check(rc, "plx_kv_quantize_fp8")
    return codes, scales


def decode_fp8kv_workspace_bytes(B: int, H: int, Hkv: int, L: int, d: int) -> int:
    return int(lib.plx_decode_fp8kv_workspace_bytes(B, H, Hkv, L, d))


def decode_fp8kv(q, r, Kcodes, Kscales, Vcodes, Vscales, seqlens, out=None, workspace=None, stream=None):
    """Decode over an e4m3 cache: q, r bf16 [B, H, d]; codes uint8 [B, Hkv, L, d];
    scales float32 [B, Hkv, L]; seqlens int32 [B]."""
    B, H, d = q.shape
    Hkv, L = Kcodes.shape[1], Kcodes.shape[2]
    if out is None:
        out = torch.empty_like(q)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()
    rc = lib.plx_decode_fp8kv(_dev(q, "q"), _dev(r, "r"), _dev(Kcodes, "Kcodes"), _dev(Kscales, "Kscales"),
                              _dev(Vcodes, "Vcodes"), _dev(Vscales, "Vscales"), _dev(seqlens, "seqlens"),
                              _dev(out, "out"), B, H, Hkv, L, d, ws_ptr, ws_bytes, _stream_ptr(stream))
    _check(rc, "plx_decode_fp8kv")
    return out


def _elsewhere(first, stream):
    """Context in which a call on the tensor ``first`` has to run: the given stream, or the tensor's device where that
    is not the current one (so that what is allocated inside may be used at once); None where both are current."""
    index = first.get_device()
    if index < 0:
        raise ValueError("tensors must be CUDA tensors")
    if stream is not None:
        if stream.device_index != index:
            raise ValueError(f"the stream is on device {stream.device_index}, the tensors on {index}")
        return torch.cuda.stream(stream)
    return None if index == torch.cuda.current_device() else torch.cuda.device(index)


def _ptr(t, name: str, shape, dtype, index: int) -> int:
    """Address of a contiguous tensor of this shape and type on device ``index``."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the other tensors on cuda:{index}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _workspace(given, need: int, index: int):
    """(tensor that keeps it alive, address, bytes) of the caller's workspace or a new one."""
    if given is None:
        if need == 0:
            return None, None, 0
        given = torch.empty(need, dtype=torch.uint8, device=index)
    elif given.get_device() != index or not given.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on cuda:{index}")
    return given, given.data_ptr(), given.numel() * given.element_size()


@functools.lru_cache(maxsize=256)
def _bytes_needed(query: str, index: int, *sizes) -> int:
    """Workspace of a call of these sizes on device ``index`` (the current one), by the entry point that tells it."""
    return getattr(lib, query)(*sizes)


_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream of a device, as its address
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def kv_quantize_int4(X, codes=None, params=None, stream=None):
    """4-bit rows of bf16 cache rows X [..., d]: returns (codes uint8 [..., d/2], params bf16 [..., 2]),
    each row standing for scale * (code - zero point) with (scale, zero point) its params."""
    at = _elsewhere(X, stream)
    if at is not None:
        with at:
            return kv_quantize_int4(X, codes, params)
    index, shape = X.get_device(), X.shape
    d, lead = shape[-1], shape[:-1]
    half, pair = (*lead, d // 2), (*lead, 2)
    if codes is None:
        codes = torch.empty(half, dtype=_U8, device=index)
    if params is None:
        params = torch.empty(pair, dtype=_BF16, device=index)
    rc = lib.plx_kv_quantize_int4(_ptr(X, "X", shape, _BF16, index), _ptr(codes, "codes", half, _U8, index),
                                  _ptr(params, "params", pair, _BF16, index), math.prod(lead), d, _raw_stream(index))
    _check(rc, "plx_kv_quantize_int4")
    return codes, params


def kv_dequantize_int4(codes, params, out=None, stream=None):
    """The bf16 values [..., d] that 4-bit rows stand for: codes uint8 [..., d/2], params bf16 [..., 2]."""
    at = _elsewhere(codes, stream)
    if at is not None:
        with at:
            return kv_dequantize_int4(codes, params, out)
    index, shape = codes.get_device(), codes.shape
    d, lead = 2 * shape[-1], shape[:-1]
    full = (*lead, d)
    if out is None:
        out = torch.empty(full, dtype=_BF16, device=index)
    rc = lib.plx_kv_dequantize_int4(_ptr(codes, "codes", shape, _U8, index),
                                    _ptr(params, "params", (*lead, 2), _BF16, index),
                                    _ptr(out, "out", full, _BF16, index), math.prod(lead), d, _raw_stream(index))
    _check(rc, "plx_kv_dequantize_int4")
    return out


def _int4_cache(Kcodes, Kparams, Vcodes, Vparams, B, Hkv, L, d, index):
    rows, words = (B, Hkv, L, d // 2), (B, Hkv, L, 2)
    return (_ptr(Kcodes, "Kcodes", rows, _U8, index), _ptr(Kparams, "Kparams", words, _BF16, index),
            _ptr(Vcodes, "Vcodes", rows, _U8, index), _ptr(Vparams, "Vparams", words, _BF16, index))


def kv_append_int4(k, v, Kcodes, Kparams, Vcodes, Vparams, seqlens, k_out=None, v_out=None, stream=None):
    """Writes the new rows k, v bf16 [B, Hkv, d] to row seqlens - 1 of a 4-bit cache (codes uint8
    [B, Hkv, L, d/2], params bf16 [B, Hkv, L, 2]); k_out, v_out, if given, get the values they stand for."""
    at = _elsewhere(k, stream)
    if at is not None:
        with at:
            return kv_append_int4(k, v, Kcodes, Kparams, Vcodes, Vparams, seqlens, k_out, v_out)
    index, new = k.get_device(), k.shape
    B, Hkv, d = new
    L = Kcodes.shape[2]
    rc = lib.plx_kv_append_int4(_ptr(k, "k", new, _BF16, index), _ptr(v, "v", new, _BF16, index),
                                *_int4_cache(Kcodes, Kparams, Vcodes, Vparams, B, Hkv, L, d, index),
                                _ptr(seqlens, "seqlens", (B,), _I32, index),
                                None if k_out is None else _ptr(k_out, "k_out", new, _BF16, index),
                                None if v_out is None else _ptr(v_out, "v_out", new, _BF16, index),
                                B, Hkv, L, d, _raw_stream(index))
    _check(rc, "plx_kv_append_int4")


def decode_int4kv_workspace_bytes(B: int, H: int, Hkv: int, L: int, d: int) -> int:
    return int(lib.plx_decode_int4kv_workspace_bytes(B, H, Hkv, L, d))


def decode_int4kv(q, r, Kcodes, Kparams, Vcodes, Vparams, seqlens, out=None, workspace=None, stream=None):
    """Decode over a 4-bit cache: q, r bf16 [B, H, d]; codes uint8 [B, Hkv, L, d/2]; params bf16
    [B, Hkv, L, 2]; seqlens int32 [B]."""
    at = _elsewhere(q, stream)
    if at is not None:
        with at:
            return decode_int4kv(q, r, Kcodes, Kparams, Vcodes, Vparams, seqlens, out, workspace)
    index, heads = q.get_device(), q.shape
    B, H, d = heads
    _, Hkv, L, _ = Kcodes.shape
    if out is None:
        out = torch.empty_like(q)
    ws, ws_ptr, ws_bytes = _workspace(
        workspace, _bytes_needed("plx_decode_int4kv_workspace_bytes", index, B, H, Hkv, L, d), index)
    rc = lib.plx_decode_int4kv(_ptr(q, "q", heads, _BF16, index), _ptr(r, "r", heads, _BF16, index),
                               *_int4_cache(Kcodes, Kparams, Vcodes, Vparams, B, Hkv, L, d, index),
                               _ptr(seqlens, "seqlens", (B,), _I32, index), _ptr(out, "out", heads, _BF16, index),
                               B, H, Hkv, L, d, ws_ptr, ws_bytes, _raw_stream(index))
    _check(rc, "plx_decode_int4kv")
    return out


def decode_weights_workspace_bytes(B: int, H: int, Hkv: int, L: int, d: int) -> int:
    return int(lib.plx_decode_weights_workspace_bytes(B, H, Hkv, L, d))


def decode_weights(q, r, Kcache, Vcache, seqlens, weights, weights_out=None, out=None, workspace=None, stream=None):
    """decode_gqa that also writes weights_out = weights + every visible key's softmax weight, summed over
    the query heads of its KV head (fp32 [B, Hkv, L]; weights itself when None); returns out."""
    at = _elsewhere(q, stream)
    if at is not None:
        with at:
            return decode_weights(q, r, Kcache, Vcache, seqlens, weights, weights_out, out, workspace)
    index, heads, cache = q.get_device(), q.shape, Kcache.shape
    B, Hkv, L, d = cache
    H = heads[1]
    heads, totals = (B, H, d), (B, Hkv, L)
    if out is None:
        out = torch.empty_like(q)
    if weights_out is None:
        weights_out = weights
    ws, ws_ptr, ws_bytes = _workspace(
        workspace, _bytes_needed("plx_decode_weights_workspace_bytes", index, B, H, Hkv, L, d), index)
    rc = lib.plx_decode_weights(_ptr(q, "q", heads, _BF16, index), _ptr(r, "r", heads, _BF16, index),
                                _ptr(Kcache, "Kcache", cache, _BF16, index),
                                _ptr(Vcache, "Vcache", cache, _BF16, index),
                                _ptr(seqlens, "seqlens", (B,), _I32, index),
                                _ptr(weights, "weights", totals, _F32, index),
                                _ptr(weights_out, "weights_out", totals, _F32, index),
                                _ptr(out, "out", heads, _BF16, index), B, H, Hkv, L, d, ws_ptr, ws_bytes,
                                _raw_stream(index))
    _check(rc, "plx_decode_weights")
    return out


def decode_int4kv_weights(q, r, Kcodes, Kparams, Vcodes, Vparams, seqlens, weights, weights_out=None, out=None,
                          workspace=None, stream=None):
    """decode_weights over a 4-bit cache (decode_int4kv)."""
    at = _elsewhere(q, stream)
    if at is not None:
        with at:
            return decode_int4kv_weights(q, r, Kcodes, Kparams, Vcodes, Vparams, seqlens, weights, weights_out, out,
                                         workspace)
    index, heads = q.get_device(), q.shape
    B, H, d = heads
    _, Hkv, L, _ = Kcodes.shape
    totals = (B, Hkv, L)
    if out is None:
        out = torch.empty_like(q)
    if weights_out is None:
        weights_out = weights
    ws, ws_ptr, ws_bytes = _workspace(
        workspace, _bytes_needed("plx_decode_weights_workspace_bytes", index, B, H, Hkv, L, d), index)
    rc = lib.plx_decode_int4kv_weights(_ptr(q, "q", heads, _BF16, index), _ptr(r, "r", heads, _BF16, index),
                                       *_int4_cache(Kcodes, Kparams, Vcodes, Vparams, B, Hkv, L, d, index),
                                       _ptr(seqlens, "seqlens", (B,), _I32, index),
                                       _ptr(weights, "weights", totals, _F32, index),
                                       _ptr(weights_out, "weights_out", totals, _F32, index),
                                       _ptr(out, "out", heads, _BF16, index), B, H, Hkv, L, d, ws_ptr, ws_bytes,
                                       _raw_stream(index))
    _check(rc, "plx_decode_int4kv_weights")
    return out


def cache_evict(caches, weights, seqlens, budget: int, sinks: int = 0, recent: int = 0, caches_out=None,
                weights_out=None, seqlens_out=None, stream=None):
    """Cuts every sequence longer than ``budget`` to its first ``sinks`` rows, its last ``recent`` rows and the
    rows of largest weight between them, for each KV head on its own.

    caches: tensors [B, Hkv, L, ...] of any type (keys, values, codes, params, scales); weights fp32
    [B, Hkv, L]; seqlens int32 [B].  Rows move, in the order of their positions, to caches_out
    [B, Hkv, L_out, ...] and weights_out [B, Hkv, L_out] (0 behind the last), L_out >= min(budget, L); both in
    place when None.  Returns (kept int32 [B, Hkv, min(budget, L)], the rows' old positions, -1 behind the
    last; new seqlens int32 [B])."""
    at = _elsewhere(weights, stream)
    if at is not None:
        with at:
            return cache_evict(caches, weights, seqlens, budget, sinks, recent, caches_out, weights_out, seqlens_out)
    if (caches_out is None) != (weights_out is None):
        raise ValueError("caches_out and weights_out go together: both given, or both None (in place)")
    if caches_out is None:
        caches_out, weights_out = caches, weights
    if len(caches_out) != len(caches):
        raise ValueError("caches_out must hold one tensor for each of caches")
    index, (B, Hkv, L), L_out = weights.get_device(), weights.shape, weights_out.shape[-1]
    # ctypes passes the low 32 bits of larger numbers.
    if max(budget, sinks, recent, B, Hkv, L, L_out) >= 1 << 31 or min(budget, sinks, recent) < -(1 << 31):
        raise ValueError("sizes, budget, sinks and recent must fit 32 bits")
    kept = torch.empty((B, Hkv, min(max(budget, 0), L)), dtype=_I32, device=index)
    if seqlens_out is None:
        seqlens_out = torch.empty((B,), dtype=_I32, device=index)
    n = len(caches)
    src, dst, row = (_vp * n)(), (_vp * n)(), (_i * n)()
    for i, (t, o) in enumerate(zip(caches, caches_out)):
        rest = t.shape[3:]
        src[i] = _ptr(t, "caches", (B, Hkv, L, *rest), t.dtype, index)
        dst[i] = _ptr(o, "caches_out", (B, Hkv, L_out, *rest), t.dtype, index)
        row[i] = min(t.element_size() * math.prod(rest), 1 << 30)  # (refused from 65537 on)
    rc = lib.plx_cache_evict(n, src, dst, row, _ptr(weights, "weights", (B, Hkv, L), _F32, index),
                             _ptr(weights_out, "weights_out", (B, Hkv, L_out), _F32, index),
                             _ptr(seqlens, "seqlens", (B,), _I32, index),
                             _ptr(seqlens_out, "seqlens_out", (B,), _I32, index), kept.data_ptr(), B, Hkv, L, L_out,
                             budget, sinks, recent, _raw_stream(index))
    _check(rc, "plx_cache_evict")
    return kept, seqlens_out


def qkr_norm_rope(x, H: int, eps: float = 1e-6, base: float = 10000.0, out=None, stream=None):
    """x bf16 [B, N, H*d] -> RoPE(RMSNorm(.)) per head as [B, H, N, d]."""
    B, N, D = x.shape
    d = D // H
    if out is None:
        out = torch.empty((B, H, N, d), dtype=x.dtype, device=x.device)
    rc = lib.plx_qkr_norm_rope(_dev(x, "x"), _dev(out, "out"), B, N, H, d, eps, base,
                               _stream_ptr(stream))
    _check(rc, "plx_qkr_norm_rope")
    return out


def layer_forward(x, WQ, WK, WV, WR, WO, H: int, out=None, workspace=None, stream=None):
    """Full Parallax attention layer: x bf16 [B, N, H*d], W* bf16 [H*d, H*d] stored [in, out]."""
    B, N, D = x.shape
    d = D // H
    if out is None:
        out = torch.empty_like(x)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()
    rc = lib.plx_layer_forward(_dev(x, "x"), _dev(WQ, "WQ"), _dev(WK, "WK"), _dev(WV, "WV"),
                               _dev(WR, "WR"), _dev(WO, "WO"), _dev(out, "out"), B, N, H, d,
                               ws_ptr, ws_bytes, _stream_ptr(stream))
    _check(rc, "plx_layer_forward")
    return out


def layer_workspace_bytes(B: int, N: int, H: int, d: int) -> int:
    return int(lib.plx_layer_workspace_bytes(B, N, H, d))


def layer_workspace_views(workspace, B: int, N: int, H: int, d: int) -> dict:
    """Views of a caller workspace after plx_layer_forward returned: the layer's
    own bf16 attention inputs q, k, v, rho and its attention output, each
    [B, H, N, d] (the slots the header lists)."""
    slot = -(-(B * N * H * d * 2) // 256) * 256
    assert workspace.dtype == torch.uint8 and workspace.numel() >= 9 * slot
    def view(i):
        return workspace[i * slot:i * slot + B * N * H * d * 2].view(torch.bfloat16).view(B, H, N, d)
    return {"q": view(4), "k": view(5), "v": view(6), "rho": view(7), "attn": view(8)}


def layer_forward_fp8(x, WQ, WK, WV, WR, WO, H: int, out=None, workspace=None, stream=None):
    """The layer of layer_forward with its five linears in dynamic per-tensor fp8 (e4m3)."""
    B, N, D = x.shape
    d = D // H
    if out is None:
        out = torch.empty_like(x)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()
    rc = lib.plx_layer_forward_fp8(_dev(x, "x"), _dev(WQ, "WQ"), _dev(WK, "WK"), _dev(WV, "WV"),
                                   _dev(WR, "WR"), _dev(WO, "WO"), _dev(out, "out"), B, N, H, d,
                                   ws_ptr, ws_bytes, _stream_ptr(stream))
    _check(rc, "plx_layer_forward_fp8")
    return out


def get_device_status(stream=None) -> int:
    """Synchronises the stream, returns and clears the device status code."""
    return int(lib.plx_get_device_status(_stream_ptr(stream)))
