"""The tied embedding: rows of the output matrix for given tokens, and the gradient they send back to it.

Argument marshalling only, as in the package itself: every step runs in the CUDA library.

    x = fckl.embedding(W, tokens, scale=d ** 0.5)                     # [*tokens.shape, d], W's type
    dW = fckl.embedding_backward(g, tokens, V, scale=d ** 0.5)        # fp32 [V, d], zeros where unused
    fckl.embedding_backward(g, tokens, V, dW=dW, accumulate=True)     # added to the loss's dW: tied weights
    x = fckl.differentiable_embedding(W, tokens)                      # autograd

``W [V, d]`` is bf16, fp16 or fp32 (rows may lie apart); ``tokens`` are int32 of any shape, -1 marks an
empty slot (a row of zeros, no gradient). ``stream`` and CUDA graph capture: as for the scoring calls
(under capture call embedding_backward rather than autograd).
"""
from __future__ import annotations

import ctypes
import weakref

import chunked_kl_loss_gb300 as _pkg
from .scoring import _for_stream, _here, _here_all, _on_device, _rows, _stream, _value_code, _ws

__all__ = ["embedding", "embedding_backward", "differentiable_embedding"]


def _set_argtypes(lib):
    c = ctypes
    vp, i64, i32, sz, f32 = c.c_void_p, c.c_int64, c.c_int, c.c_size_t, c.c_float
    lib.fckl_embedding.restype = i32
    lib.fckl_embedding.argtypes = [vp, i32, i64, vp, i64, i32, i32, f32, vp, i64, vp, sz, vp]
    lib.fckl_embedding_backward_workspace_bytes.restype = sz
    lib.fckl_embedding_backward_workspace_bytes.argtypes = [i64, i32, i32]
    lib.fckl_embedding_backward.restype = i32
    lib.fckl_embedding_backward.argtypes = [vp, i32, i64, vp, i64, i32, i32, f32, vp, i32, i32, vp, sz, vp]


def _tokens(tokens):
    import torch
    if tokens.dtype is not torch.int32:
        raise TypeError(f"tokens must be {torch.int32}, got {tokens.dtype}")
    if not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous")
    return tokens.numel()


def _row_matrix(name, t, tokens, d):
    """(row pitch) of a tensor [*tokens.shape, d]: contiguous, or for tokens [N] with rows apart."""
    if tuple(t.shape) != (*tokens.shape, d):
        raise ValueError(f"{name} must be of shape {[*tokens.shape, d]}, got {list(t.shape)}")
    if t.is_contiguous():
        return d
    if t.dim() != 2:
        raise ValueError(f"{name} must be contiguous")
    return _rows(name, t)


def embedding(W, tokens, scale=1.0, out=None, ws=None, stream=None):
    """``scale`` times the rows of W [V, d] for ``tokens`` (int32, any shape): [*tokens.shape, d] of W's
    type, the product in fp32 and rounded once. An empty slot (-1) gives zeros; an id outside [0, V) is
    reported by check() (its row is NaN)."""
    import torch
    if W.dim() != 2:
        raise ValueError("expected W [V,d]")
    code = _value_code(W, "W")
    V, d = W.shape
    N = _tokens(tokens)
    ldw = d if W.is_contiguous() else _rows("W", W)
    dev = W.device
    given = out is not None
    if given:
        if out.dtype != W.dtype:
            raise TypeError(f"out must be {W.dtype}, got {out.dtype}")
        ldo = _row_matrix("out", out, tokens, d)
    if not _here_all(W, tokens, out):
        _on_device(dev, W=W, tokens=tokens, out=out)
    with _here if stream is None else _for_stream(stream, W, tokens, out, ws):
        ws = _ws(ws, dev)
        if out is None:
            out, ldo = torch.empty(*tokens.shape, d, dtype=W.dtype, device=dev), d
    st = _pkg.load().fckl_embedding(W.data_ptr(), code, ldw, tokens.data_ptr(), N, d, V, float(scale), out.data_ptr(), ldo,
                                    ws.tensor.data_ptr(), ws.nbytes, _stream(stream))
    if st != _pkg.OK:
        raise _pkg.FcklError(st, "fckl_embedding")
    if given:
        torch.autograd.graph.increment_version(out)  # a backward pass that saved it raises
    return out


def embedding_backward(g, tokens, V, scale=1.0, dW=None, accumulate=False, dtype=None, ws=None, stream=None):
    """dW [V, d] of the rows' gradients g [*tokens.shape, d]: ``scale`` times the sum of g over each token's
    positions, zeros for tokens that do not occur. ``dtype``: fp32 (the default) or g's type, rounded once
    from the fp32 sums. ``dW``: where it goes; with ``accumulate`` it is added to what is there, and only
    the rows of tokens that occur are touched. ``ws``: Workspace(N, d, V, 0, 0, kind="embedding_backward")."""
    import torch
    code = _value_code(g, "g")
    N = _tokens(tokens)
    if g.dim() < 1:
        raise ValueError("expected g [*tokens.shape, d]")
    d = g.shape[-1]
    ldg = _row_matrix("g", g, tokens, d)
    if accumulate and dW is None:
        raise ValueError("accumulate needs the dW that is added to")
    given = dW is not None
    if given:
        if dtype not in (None, dW.dtype):
            raise TypeError(f"dW must be {dtype}, got {dW.dtype}")
        if tuple(dW.shape) != (V, d) or not dW.is_contiguous():
            raise ValueError(f"dW must be contiguous of shape {[V, d]}, got {list(dW.shape)}")
        dtype = dW.dtype
    dtype = dtype or torch.float32
    if dtype not in (torch.float32, g.dtype):
        raise TypeError(f"dW is float32 or of g's type, not {dtype}")
    dev = g.device
    if not _here_all(g, tokens, dW):
        _on_device(dev, g=g, tokens=tokens, dW=dW)
    with _here if stream is None else _for_stream(stream, g, tokens, dW, ws):
        if dW is None:
            dW = torch.empty(V, d, dtype=dtype, device=dev)
        _backward(g, code, ldg, tokens, N, d, V, scale, dW, accumulate, ws, stream)
    if given:
        torch.autograd.graph.increment_version(dW)  # a backward pass that saved it raises
    return dW


def _backward(g, code, ldg, tokens, N, d, V, scale, dW, accumulate=False, ws=None, stream=None):
    """embedding_backward of checked arguments, into dW."""
    lib = _pkg.load()
    if ws is None:
        n = lib.fckl_embedding_backward_workspace_bytes(N, d, V)
        if n == 0:
            raise _pkg.FcklError(_pkg.ERR_UNSUPPORTED, "workspace_bytes")
        ws = _pkg._last_ws = _pkg.Workspace.sized(n, g.device)
    else:
        _pkg._last_ws = weakref.ref(ws)
    st = lib.fckl_embedding_backward(g.data_ptr(), code, ldg, tokens.data_ptr(), N, d, V, float(scale), dW.data_ptr(),
                                     _value_code(dW, "dW"), int(bool(accumulate)), ws.tensor.data_ptr(), ws.nbytes,
                                     _stream(stream))
    if st != _pkg.OK:
        raise _pkg.FcklError(st, "fckl_embedding_backward")


def _autograd_function():
    import torch

    class Embedding(torch.autograd.Function):
        @staticmethod
        def forward(ctx, W, tokens, scale):
            ctx.save_for_backward(tokens)
            ctx.shape = (W.shape, W.dtype, scale)
            return embedding(W, tokens, scale)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, g):
            tokens, = ctx.saved_tensors
            (V, d), dtype, scale = ctx.shape
            dW = torch.empty(V, d, dtype=dtype, device=g.device)
            _backward(g.contiguous(), _value_code(g, "g"), d, tokens, tokens.numel(), d, V, scale, dW)
            return dW, None, None

    return Embedding


_Embedding = None


def differentiable_embedding(W, tokens, scale=1.0):
    """``embedding``, differentiable in W (its gradient is summed in fp32 and rounded once to W's type)."""
    global _Embedding
    if _Embedding is None:
        _Embedding = _autograd_function()
    return _Embedding.apply(W, tokens, float(scale))
