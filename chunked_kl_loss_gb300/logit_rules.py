"""Logits adjusted by a request's rules before they are scored or sampled from: penalties for repeated
tokens, biases and masks of allowed tokens, with the gradient.

Argument marshalling only, as in the package itself: every step runs in the CUDA library.

    z = fckl.adjust_logits(logits, history, lengths, prompt, repetition=1.1, frequency=0.2, allowed=bits)
    logp, entropy, norm, _, _ = fckl.token_logprobs(z, tokens)
    dz = fckl.token_logprobs_backward(z, tokens, norm, entropy, g_logp)
    dlogits = fckl.adjust_logits_backward(dz, logits, history, lengths, repetition=1.1, allowed=bits)
    z = fckl.differentiable_adjusted_logits(logits, history, lengths, repetition=1.1)      # autograd

``logits [N, V]`` are bf16, fp16 or fp32 (rows may lie apart). ``history [N, L]`` int32 holds each row's
tokens so far: its first ``lengths[n]`` entries, of which the first ``prompt[n]`` were given and the others
generated; -1 is an empty slot. Penalties are numbers, or fp32 tensors [N]. ``allowed`` is int32
[N, ceil(V / 32)] (or [ceil(V / 32)], the same for all rows): bit v % 32 of word v // 32 allows token v.
"""
from __future__ import annotations

import ctypes

import chunked_kl_loss_gb300 as _pkg
from .scoring import _address, _dense, _for_stream, _here, _here_all, _on_device, _rows, _stream, _value_code, _ws

__all__ = ["adjust_logits", "adjust_logits_backward", "differentiable_adjusted_logits"]


def _set_argtypes(lib):
    c = ctypes
    vp, i64, i32, sz, f32 = c.c_void_p, c.c_int64, c.c_int, c.c_size_t, c.c_float
    lib.fckl_adjust_logits.restype = i32
    lib.fckl_adjust_logits.argtypes = [vp, i32, i64, i64, i32, vp, i64, i32, vp, vp, vp, f32, vp, f32, vp, f32, vp, vp,
                                       i32, vp, i64, vp, i64, vp, sz, vp]
    lib.fckl_adjust_logits_backward.restype = i32
    lib.fckl_adjust_logits_backward.argtypes = [vp, i32, i64, vp, i64, i64, i32, vp, i64, i32, vp, vp, f32, vp, i64, vp,
                                                i64, vp, sz, vp]


def _history(history, lengths, prompt, N):
    """(row pitch, L) of the history."""
    import torch
    if history is None:
        if lengths is not None or prompt is not None:
            raise ValueError("lengths and prompt need a history")
        return 0, 0
    if history.dtype != torch.int32:
        raise TypeError(f"history must be {torch.int32}, got {history.dtype}")
    if history.dim() != 2 or history.shape[0] != N:
        raise ValueError(f"expected history [{N}, L], got {list(history.shape)}")
    for name, t in (("lengths", lengths), ("prompt", prompt)):
        if t is not None:
            _dense(name, t, torch.int32, (N,))
    return _rows("history", history), history.shape[1]


def _penalty(name, value, N):
    """(tensor or None, number) of a penalty."""
    import torch
    if isinstance(value, torch.Tensor):
        _dense(name, value, torch.float32, (N,))
        return value, 0.0
    return None, float(value)


def _bits(allowed, N, V):
    """Row pitch, in words, of the bits of allowed tokens (0: one row for all)."""
    import torch
    if allowed is None:
        return 0
    words = -(-V // 32)
    if allowed.dtype != torch.int32:
        raise TypeError(f"allowed must be {torch.int32}, got {allowed.dtype}")
    if tuple(allowed.shape) not in ((words,), (N, words)):
        raise ValueError(f"allowed must be [{N}, {words}] or [{words}], got {list(allowed.shape)}")
    if words > 1 and allowed.stride(-1) != 1:
        raise ValueError("allowed must be dense in its last dimension")
    if allowed.dim() == 1 or N == 1 or allowed.stride(0) == 0:
        return 0
    if allowed.stride(0) < words:
        raise ValueError("allowed: rows must not overlap")
    return allowed.stride(0)


def _out(out, like):
    """Row pitch of `out`."""
    if out.dtype != like.dtype or out.shape != like.shape:
        raise ValueError("out must have the logits' type and shape")
    return _rows("out", out)


def adjust_logits(logits, history=None, lengths=None, prompt=None, repetition=1.0, frequency=0.0, presence=0.0,
                  bias_tokens=None, bias=None, allowed=None, out=None, ws=None, stream=None):
    """Logits [N, V] under each row's rules, of the logits' type. A token of the history: z / repetition
    where z > 0, else z * repetition; a generated one: less frequency times its number and less presence;
    then the sum of its biases (``bias_tokens`` int32 [N, B], -1 empty, and ``bias`` fp32 [N, B]); -inf
    where it is not allowed. ``out`` may be ``logits``: without a mask only what a rule changes is then
    touched. An id outside [-1, V) is skipped and reported by check()."""
    import torch
    if logits.dim() != 2:
        raise ValueError("expected logits [N,V]")
    code = _value_code(logits, "logits")
    N, V = logits.shape
    ld = _rows("logits", logits)
    ldh, L = _history(history, lengths, prompt, N)
    r, r1 = _penalty("repetition", repetition, N)
    f, f1 = _penalty("frequency", frequency, N)
    p, p1 = _penalty("presence", presence, N)
    if r is None and not r1 > 0:
        raise ValueError(f"repetition must be positive, got {r1}")
    B = 0
    if (bias_tokens is None) != (bias is None):
        raise ValueError("bias_tokens and bias go together")
    if bias is not None:
        if bias_tokens.dim() != 2:
            raise ValueError("expected bias_tokens [N,B]")
        B = bias_tokens.shape[1]
        _dense("bias_tokens", bias_tokens, torch.int32, (N, B))
        _dense("bias", bias, torch.float32, (N, B))
    lda = _bits(allowed, N, V)
    ldo, given = V, out is not None
    if given:
        ldo = _out(out, logits)
    dev = logits.device
    if not _here_all(logits, history, lengths, prompt, r, f, p, bias_tokens, bias, allowed, out):
        _on_device(dev, logits=logits, history=history, lengths=lengths, prompt=prompt, repetition=r, frequency=f,
                   presence=p, bias_tokens=bias_tokens, bias=bias, allowed=allowed, out=out)
    used = (logits, history, lengths, prompt, r, f, p, bias_tokens, bias, allowed, out, ws)
    with _here if stream is None else _for_stream(stream, *used):
        ws = _ws(ws, dev)
        if out is None:
            out = torch.empty(N, V, dtype=logits.dtype, device=dev)
    a = _address
    st = _pkg.load().fckl_adjust_logits(a(logits), code, ld, N, V, a(history), ldh, L, a(lengths), a(prompt), a(r), r1, a(f),
                                        f1, a(p), p1, a(bias_tokens), a(bias), B, a(allowed), lda, a(out),
                                        ldo, ws.tensor.data_ptr(), ws.nbytes, _stream(stream))
    if st != _pkg.OK:
        raise _pkg.FcklError(st, "fckl_adjust_logits")
    if given:
        torch.autograd.graph.increment_version(out)  # a backward pass that saved it raises
    return out


def adjust_logits_backward(g, logits, history=None, lengths=None, repetition=1.0, allowed=None, out=None, ws=None,
                           stream=None):
    """Gradient [N, V] with respect to the logits that went into adjust_logits, of the upstream gradient g
    [N, V] (of the logits' type): times the repetition penalty's slope at the history's tokens, 0 where a
    token is not allowed. ``out`` may be ``g``: without a mask only what changes is then touched."""
    import torch
    if logits.dim() != 2 or g.shape != logits.shape:
        raise ValueError("expected logits [N,V] and g [N,V]")
    if g.dtype != logits.dtype:
        raise TypeError("g and logits must share a dtype")
    code = _value_code(logits, "logits")
    N, V = logits.shape
    ldg, ld = _rows("g", g), _rows("logits", logits)
    ldh, L = _history(history, lengths, None, N)
    r, r1 = _penalty("repetition", repetition, N)
    if r is None and not r1 > 0:
        raise ValueError(f"repetition must be positive, got {r1}")
    lda = _bits(allowed, N, V)
    ldo, given = V, out is not None
    if given:
        ldo = _out(out, logits)
    dev = logits.device
    if not _here_all(logits, g, history, lengths, r, allowed, out):
        _on_device(dev, logits=logits, g=g, history=history, lengths=lengths, repetition=r, allowed=allowed, out=out)
    with _here if stream is None else _for_stream(stream, g, logits, history, lengths, r, allowed, out, ws):
        ws = _ws(ws, dev)
        if out is None:
            out = torch.empty(N, V, dtype=logits.dtype, device=dev)
    a = _address
    st = _pkg.load().fckl_adjust_logits_backward(a(g), code, ldg, a(logits), ld, N, V, a(history), ldh, L, a(lengths), a(r),
                                                 r1, a(allowed), lda, a(out), ldo, ws.tensor.data_ptr(),
                                                 ws.nbytes, _stream(stream))
    if st != _pkg.OK:
        raise _pkg.FcklError(st, "fckl_adjust_logits_backward")
    if given:
        torch.autograd.graph.increment_version(out)  # a backward pass that saved it raises
    return out


def _autograd_function():
    import torch

    class AdjustedLogits(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, history, lengths, prompt, repetition, frequency, presence, bias_tokens, bias, allowed):
            tensor = isinstance(repetition, torch.Tensor)
            ctx.save_for_backward(logits, history, lengths, repetition if tensor else None, allowed)
            ctx.repetition = None if tensor else repetition
            return adjust_logits(logits, history, lengths, prompt, repetition, frequency, presence, bias_tokens, bias,
                                 allowed)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, g):
            logits, history, lengths, r, allowed = ctx.saved_tensors
            if r is None:
                r = ctx.repetition
            return (adjust_logits_backward(g.contiguous(), logits, history, lengths, r, allowed),) + (None,) * 9

    return AdjustedLogits


_AdjustedLogits = None


def differentiable_adjusted_logits(logits, history=None, lengths=None, prompt=None, repetition=1.0, frequency=0.0,
                                   presence=0.0, bias_tokens=None, bias=None, allowed=None):
    """``adjust_logits``, differentiable in the logits. Penalties and biases have no gradient: one that
    requires it is refused (detach it)."""
    import torch
    global _AdjustedLogits
    if torch.is_grad_enabled():
        for name, t in (("repetition", repetition), ("frequency", frequency), ("presence", presence), ("bias", bias)):
            if isinstance(t, torch.Tensor) and t.requires_grad:
                raise ValueError(f"{name} has no gradient: detach it")
    if _AdjustedLogits is None:
        _AdjustedLogits = _autograd_function()
    return _AdjustedLogits.apply(logits, history, lengths, prompt, repetition, frequency, presence, bias_tokens, bias,
                                 allowed)
