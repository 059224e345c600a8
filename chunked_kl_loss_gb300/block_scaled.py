"""Output projection in 8-bit floating point (e4m3) with a scale for each block of 128.

Argument marshalling only, as in the package itself: every step runs in the CUDA library.

    W8, w_scale = fckl.block_quantize(W, rows=128)                 # once per checkpoint
    logits = fckl.block_scaled_projection(H, W8, w_scale)           # H quantised on the way in
    H8, h_scale = fckl.block_quantize(H)                            # or step by step
    logits = fckl.block_scaled_matmul(H8, h_scale, W8, w_scale)

An 8-bit tensor is float8_e4m3fn [R, K] whose rows start on 16-byte boundaries; its scales are fp32
[ceil(R / rows), ceil(K / 128)], one per block of ``rows`` x 128 values, in any layout. There is no
gradient: the 8-bit head is a teacher's.
"""
from __future__ import annotations

import ctypes

import chunked_kl_loss_gb300 as _pkg
from .scoring import _address, _for_stream, _on_device, _rows, _stream, _value_code, _ws

__all__ = ["block_quantize", "block_scaled_matmul", "block_scaled_projection"]

BLOCK = 128


def _set_argtypes(lib):
    c = ctypes
    vp, i64, i32, sz = c.c_void_p, c.c_int64, c.c_int, c.c_size_t
    lib.fckl_block_quantize.restype = i32
    lib.fckl_block_quantize.argtypes = [vp, i32, i64, i64, i64, i32, vp, i64, vp, i64, i64, vp]
    lib.fckl_block_scaled_matmul.restype = i32
    lib.fckl_block_scaled_matmul.argtypes = [vp, i64, vp, i64, i64, vp, i64, vp, i64, i64, i64, i64, i64, vp, i32, i64,
                                             vp, sz, vp]


def _pitch(name, q):
    """Bytes between rows of an 8-bit tensor (of one row: its own length on the next boundary)."""
    import torch
    if q.dtype != torch.float8_e4m3fn:
        raise TypeError(f"{name} must be float8_e4m3fn, got {q.dtype}")
    R, K = q.shape
    if K > 1 and q.stride(1) != 1:
        raise ValueError(f"{name} must be dense in its last dimension")
    if R <= 1:
        return -(-K // 16) * 16
    if q.stride(0) < K or q.stride(0) % 16:
        raise ValueError(f"{name}: rows must start on 16-byte boundaries and not overlap")
    return q.stride(0)


def _scale_strides(name, s, shape):
    import torch
    if s.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {s.dtype}")
    if tuple(s.shape) != tuple(shape):
        raise ValueError(f"{name} must be of shape {list(shape)}, got {list(s.shape)}")
    rs = s.stride(0) if shape[0] > 1 else 1
    cs = s.stride(1) if shape[1] > 1 else 1
    if rs < 1 or cs < 1:
        raise ValueError(f"{name} must not be broadcast")
    return rs, cs


def _out_dtype(out, out_dtype, M, N):
    import torch
    if out is not None:
        if out_dtype not in (None, out.dtype) or tuple(out.shape) != (M, N):
            raise ValueError(f"out must be [{M}, {N}] of out_dtype")
        out_dtype = out.dtype
    out_dtype = out_dtype or torch.bfloat16
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"the product is bfloat16 or float32, not {out_dtype}")
    return out_dtype


def block_quantize(x, rows=1, stream=None):
    """(e4m3 values [R, K], fp32 scales [ceil(R / rows), ceil(K / 128)]) of x [R, K] (bf16, fp16 or
    fp32): each block of ``rows`` (1 or 128) x 128 values is divided by max(amax / 448, 2^-126)."""
    import torch
    if x.dim() != 2:
        raise ValueError("expected x [R,K]")
    if rows not in (1, BLOCK):
        raise ValueError(f"rows must be 1 or {BLOCK}")
    code = _value_code(x, "x")
    R, K = x.shape
    ldx = _rows("x", x)
    _on_device(x.device, x=x)
    kb = -(-K // BLOCK)
    with _for_stream(stream, x):
        q = torch.empty(R, -(-K // 16) * 16, dtype=torch.float8_e4m3fn, device=x.device)[:, :K]
        scale = torch.empty(-(-R // rows), kb, dtype=torch.float32, device=x.device)
    p = _address
    st = _pkg.load().fckl_block_quantize(p(x), code, ldx, R, K, rows, p(q), -(-K // 16) * 16, p(scale), kb, 1,
                                         _stream(stream))
    if st != _pkg.OK:
        raise _pkg.FcklError(st, "fckl_block_quantize")
    return q, scale


def block_scaled_matmul(a, a_scale, b, b_scale, out_dtype=None, out=None, ws=None, stream=None):
    """a [M, K] times the transpose of b [N, K], both e4m3 with a_scale [M, ceil(K / 128)] and
    b_scale [ceil(N / 128), ceil(K / 128)]: [M, N] in bf16 (the default) or fp32, summed in fp32."""
    import torch
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[1]:
        raise ValueError("expected a [M,K] and b [N,K]")
    M, K = a.shape
    N = b.shape[0]
    kb = -(-K // BLOCK)
    lda, ldb = _pitch("a", a), _pitch("b", b)
    sa = _scale_strides("a_scale", a_scale, (M, kb))
    sb = _scale_strides("b_scale", b_scale, (-(-N // BLOCK), kb))
    out_dtype = _out_dtype(out, out_dtype, M, N)
    dev = a.device
    _on_device(dev, a=a, a_scale=a_scale, b=b, b_scale=b_scale, out=out)
    with _for_stream(stream, a, a_scale, b, b_scale, out, ws):
        ws = _ws(ws, dev)
        if out is None:
            out = torch.empty(M, N, dtype=out_dtype, device=dev)
    p = _address
    st = _pkg.load().fckl_block_scaled_matmul(p(a), lda, p(a_scale), *sa, p(b), ldb, p(b_scale), *sb, M, N, K, p(out),
                                              _value_code(out, "out"), _rows("out", out), ws.tensor.data_ptr(), ws.nbytes,
                                              _stream(stream))
    if st != _pkg.OK:
        raise _pkg.FcklError(st, "fckl_block_scaled_matmul")
    return out


def block_scaled_projection(H, W8, w_scale, out_dtype=None, out=None, ws=None, stream=None):
    """Logits [N, V] of hidden states H [N, K] (bf16, fp16 or fp32) against an output matrix in
    8 bits: H is quantised by position and block of 128 channels, then multiplied (block_quantize and
    block_scaled_matmul with one set of checks)."""
    import torch
    if H.dim() != 2 or W8.dim() != 2 or H.shape[1] != W8.shape[1]:
        raise ValueError("expected H [N,K] and W8 [V,K]")
    code = _value_code(H, "H")
    N, K = H.shape
    V = W8.shape[0]
    kb = -(-K // BLOCK)
    ldx, ldb = _rows("H", H), _pitch("W8", W8)
    sb = _scale_strides("w_scale", w_scale, (-(-V // BLOCK), kb))
    out_dtype = _out_dtype(out, out_dtype, N, V)
    dev = H.device
    _on_device(dev, H=H, W8=W8, w_scale=w_scale, out=out)
    ldq = -(-K // 16) * 16
    with _for_stream(stream, H, W8, w_scale, out, ws):
        ws = _ws(ws, dev)
        q = torch.empty(N * ldq, dtype=torch.uint8, device=dev)
        scale = torch.empty(N * kb, dtype=torch.float32, device=dev)
        if out is None:
            out = torch.empty(N, V, dtype=out_dtype, device=dev)
    lib, s, p = _pkg.load(), _stream(stream), _address
    st = lib.fckl_block_quantize(p(H), code, ldx, N, K, 1, p(q), ldq, p(scale), kb, 1, s)
    if st != _pkg.OK:
        raise _pkg.FcklError(st, "fckl_block_quantize")
    st = lib.fckl_block_scaled_matmul(p(q), ldq, p(scale), kb, 1, p(W8), ldb, p(w_scale), *sb, N, V, K, p(out),
                                      _value_code(out, "out"), _rows("out", out), ws.tensor.data_ptr(), ws.nbytes, s)
    if st != _pkg.OK:
        raise _pkg.FcklError(st, "fckl_block_scaled_matmul")
    return out
