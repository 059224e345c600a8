"""Scoring of given tokens: log-probabilities, entropy and most probable tokens, with gradients.

Argument marshalling only, as in the package itself: every step runs in the CUDA library.

    logp, entropy, norm, top_idx, top_logp = fckl.token_logprobs(logits, tokens, top=20)
    dlogits = fckl.token_logprobs_backward(logits, tokens, norm, entropy, g_logp, g_entropy)
    logp, entropy = fckl.differentiable_token_logprobs(logits, tokens)         # autograd
    logp, entropy, lse = fckl.projected_logprobs(H, W, tokens, chunk)           # from hidden states
    dH, dW = fckl.projected_logprobs_backward(H, W, tokens, lse, entropy, g_logp, g_entropy, chunk=chunk)
    logp, entropy = fckl.fused_token_logprobs(H, W, tokens, chunk)             # autograd

``logits [N, V]`` are bf16, fp16 or fp32 (rows may lie apart: only the last dimension has to be
dense); ``tokens [N, T]`` are int32, -1 marks an empty slot. Logits of -inf are masked tokens.
``H [N, d]`` and ``W [V, d]`` are bf16 or fp32 as for the loss; their logits are never stored.

``stream`` launches on a stream other than the current one: outputs are then allocated for that
stream, and the inputs and a workspace passed as ``ws`` are marked as used on it; making the inputs'
data ready there is the caller's part. Under CUDA graph capture call the functions that take
gradients directly rather than autograd (whose accumulation nodes remember the stream that an eager
pass used).
"""
from __future__ import annotations

import contextlib
import ctypes

import chunked_kl_loss_gb300 as _pkg

__all__ = ["token_logprobs", "token_logprobs_backward", "differentiable_token_logprobs", "projected_logprobs",
           "projected_logprobs_backward", "fused_token_logprobs"]

_status_ws = {}  # device index -> workspace that holds only a status word


def _set_argtypes(lib):
    c = ctypes
    vp, i64, i32, sz = c.c_void_p, c.c_int64, c.c_int, c.c_size_t
    lib.fckl_projected_logprobs_workspace_bytes.restype = sz
    lib.fckl_projected_logprobs_workspace_bytes.argtypes = [i64, i32, i32, i32, i32, i32, i32]
    lib.fckl_projected_logprobs.restype = i32
    lib.fckl_projected_logprobs.argtypes = [vp, vp, i32, vp, i64, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    lib.fckl_projected_logprobs_backward.restype = i32
    lib.fckl_projected_logprobs_backward.argtypes = [vp, vp, i32, vp, i64, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp,
                                                     vp, vp, sz, vp]
    lib.fckl_token_logprobs.restype = i32
    lib.fckl_token_logprobs.argtypes = [vp, i32, i64, vp, i64, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.fckl_token_logprobs_backward.restype = i32
    lib.fckl_token_logprobs_backward.argtypes = [vp, i32, i64, vp, i64, i32, i32, vp, vp, vp, vp, vp, i64, vp, sz, vp]


def _stream(stream):
    """Handle of ``stream``, or of the current stream."""
    import torch
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _status_workspace(device):
    """The device's status word: zeroed once, shared by every call that is given no workspace (the
    word only gathers bits, so calls on several streams may share it)."""
    import torch
    ws = _status_ws.get(device.index)
    if ws is None:
        ws = _pkg.Workspace.status(device)
        if torch.cuda.is_current_stream_capturing():
            return ws  # belongs to the graph being captured
        torch.cuda.current_stream(device).synchronize()  # zeroed before any stream uses it
        _status_ws[device.index] = ws
    return ws


def _ws(ws, device):
    import weakref
    if ws is None:
        ws = _status_workspace(device)
        _pkg._last_ws = ws
    else:
        _pkg._last_ws = weakref.ref(ws)
    return ws


def _value_code(t, what):
    import torch
    code = {torch.bfloat16: _pkg.BF16, torch.float16: _pkg.F16, torch.float32: _pkg.F32}.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be bfloat16, float16 or float32, got {t.dtype}")
    return code


def _on_device(device, **tensors):
    import torch
    if device.type != "cuda" or device.index != torch.cuda.current_device():
        raise ValueError(f"tensors must be on the current CUDA device, got {device}")
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}, got {t.device}")


def _dense(name, t, dtype, shape):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous of shape {list(shape)}, got {list(t.shape)}")


def _rows(name, t):
    """Row pitch of a [N, V] tensor whose rows are dense."""
    N, V = t.shape
    if V > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be dense in its last dimension")
    if N <= 1:
        return V
    if t.stride(0) < V:
        raise ValueError(f"{name}: rows must not overlap")
    return t.stride(0)


def _address(t):
    return None if t is None else t.data_ptr()


_here = contextlib.nullcontext()


def _for_stream(stream, *inputs):
    """Context for allocations that `stream` will use (None: the current stream); `inputs`, a workspace
    of the caller's among them, are marked as used there."""
    import torch
    if stream is None:
        return _here
    for t in inputs:
        if t is not None:
            (t.tensor if isinstance(t, _pkg.Workspace) else t).record_stream(stream)
    return torch.cuda.stream(stream)


def _logits_args(logits, tokens):
    import torch
    if logits.dim() != 2 or tokens.dim() != 2 or tokens.shape[0] != logits.shape[0]:
        raise ValueError("expected logits [N,V] and tokens [N,T]")
    code = _value_code(logits, "logits")
    N, V = logits.shape
    T = tokens.shape[1]
    _dense("tokens", tokens, torch.int32, (N, T))
    return code, N, V, T, _rows("logits", logits)


def token_logprobs(logits, tokens, top=0, ws=None, stream=None):
    """(logp fp32 [N, T], entropy fp32 [N], norm fp32 [N, 2], top_idx int32 [N, top],
    top_logp fp32 [N, top]) of logits [N, V]: the given tokens' log-probabilities, the entropy,
    (max z, log sum exp(z - max z)), and the ``top`` most probable tokens, largest first, equal
    ones by smaller id. An id outside [0, V) is reported by check() (its logp is NaN)."""
    import torch
    code, N, V, T, ld = _logits_args(logits, tokens)
    dev = logits.device
    _on_device(dev, logits=logits, tokens=tokens)
    f32 = torch.float32
    with _for_stream(stream, logits, tokens, ws):
        ws = _ws(ws, dev)
        logp = torch.empty(N, T, dtype=f32, device=dev)
        entropy = torch.empty(N, dtype=f32, device=dev)
        norm = torch.empty(N, 2, dtype=f32, device=dev)
        top_idx = torch.empty(N, max(top, 0), dtype=torch.int32, device=dev)
        top_logp = torch.empty(N, max(top, 0), dtype=f32, device=dev)
    p = _address
    st = _pkg.load().fckl_token_logprobs(p(logits), code, ld, p(tokens), N, V, T, top, p(logp), p(entropy), p(norm),
                                         p(top_idx), p(top_logp), ws.tensor.data_ptr(), ws.nbytes, _stream(stream))
    if st != _pkg.OK:
        raise _pkg.FcklError(st, "fckl_token_logprobs")
    return logp, entropy, norm, top_idx, top_logp


def token_logprobs_backward(logits, tokens, norm, entropy, g_logp, g_entropy=None, out=None, ws=None, stream=None):
    """Gradient [N, V], of the logits' type, of sum g_logp * logp + sum g_entropy * entropy with
    respect to the logits; ``norm`` and ``entropy`` as token_logprobs returned them. ``out`` may be
    ``logits`` itself, whose values are then lost."""
    import torch
    code, N, V, T, ld = _logits_args(logits, tokens)
    dev = logits.device
    _on_device(dev, logits=logits, tokens=tokens, norm=norm, entropy=entropy, g_logp=g_logp, g_entropy=g_entropy,
               out=out)
    f32 = torch.float32
    _dense("norm", norm, f32, (N, 2))
    _dense("entropy", entropy, f32, (N,))
    _dense("g_logp", g_logp, f32, (N, T))
    if g_entropy is not None:
        _dense("g_entropy", g_entropy, f32, (N,))
    if out is not None and (out.dtype != logits.dtype or out.shape != logits.shape):
        raise ValueError("out must have the logits' type and shape")
    with _for_stream(stream, logits, tokens, norm, entropy, g_logp, g_entropy, out, ws):
        ws = _ws(ws, dev)
        if out is None:
            out = torch.empty(N, V, dtype=logits.dtype, device=dev)
    p = _address
    st = _pkg.load().fckl_token_logprobs_backward(p(logits), code, ld, p(tokens), N, V, T, p(norm), p(entropy),
                                                  p(g_logp), p(g_entropy), p(out), _rows("out", out), ws.ptr,
                                                  ws.nbytes, _stream(stream))
    if st != _pkg.OK:
        raise _pkg.FcklError(st, "fckl_token_logprobs_backward")
    return out


def _upstream(g, shape, device):
    """An upstream gradient as the library reads it: dense fp32 (autograd hands over expanded ones)."""
    import torch
    if g is None:
        return torch.zeros(shape, dtype=torch.float32, device=device)
    return g.to(torch.float32).contiguous()


def _autograd_function():
    import torch

    class TokenLogprobs(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, tokens):
            logp, entropy, norm, _, _ = token_logprobs(logits, tokens)
            ctx.save_for_backward(logits, tokens, norm, entropy)
            ctx.set_materialize_grads(False)
            return logp, entropy

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, g_logp, g_entropy):
            logits, tokens, norm, entropy = ctx.saved_tensors
            if g_logp is None and g_entropy is None:
                return None, None
            ge = None if g_entropy is None else _upstream(g_entropy, None, logits.device)
            gl = _upstream(g_logp, tuple(tokens.shape), logits.device)
            return token_logprobs_backward(logits, tokens, norm, entropy, gl, ge), None

    return TokenLogprobs


_TokenLogprobs = None


def differentiable_token_logprobs(logits, tokens):
    """(logp [N, T], entropy [N]) of logits [N, V], differentiable in the logits."""
    global _TokenLogprobs
    if _TokenLogprobs is None:
        _TokenLogprobs = _autograd_function()
    return _TokenLogprobs.apply(logits, tokens)


# ------------------------------------------------------------------ from hidden states
def _head_args(H, W, tokens):
    import torch
    if H.dim() != 2 or W.dim() != 2 or tokens.dim() != 2 or W.shape[1] != H.shape[1] or \
            tokens.shape[0] != H.shape[0]:
        raise ValueError("expected H [N,d], W [V,d], tokens [N,T]")
    if H.dtype != W.dtype:
        raise TypeError("H and W must share a dtype")
    dt = _pkg._dtype_code(H)
    for name, t in (("H", H), ("W", W)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    N, d = H.shape
    V, T = W.shape[0], tokens.shape[1]
    _dense("tokens", tokens, torch.int32, (N, T))
    return dt, N, d, V, T


def _head_ws(ws, N, d, V, T, chunk, dt, device, backward):
    import weakref
    if ws is None:
        n = _pkg.load().fckl_projected_logprobs_workspace_bytes(N, d, V, T, chunk, dt, backward)
        if n == 0:
            raise _pkg.FcklError(_pkg.ERR_UNSUPPORTED, "workspace_bytes")
        ws = _pkg._last_ws = _pkg.Workspace.sized(n, device)
    else:
        _pkg._last_ws = weakref.ref(ws)
    return ws


def _projected(dt, N, d, V, T, H, W, tokens, chunk, ws=None, stream=None):
    """projected_logprobs of checked arguments."""
    import torch
    dev = H.device
    ws = _head_ws(ws, N, d, V, T, chunk, dt, dev, 0)
    logp = torch.empty(N, T, dtype=torch.float32, device=dev)
    entropy = torch.empty(N, dtype=torch.float32, device=dev)
    lse = torch.empty(N, dtype=torch.float32, device=dev)
    p = _address
    st = _pkg.load().fckl_projected_logprobs(p(H), p(W), dt, p(tokens), N, d, V, T, chunk, p(logp), p(entropy),
                                             p(lse), ws.tensor.data_ptr(), ws.nbytes, _stream(stream))
    if st != _pkg.OK:
        raise _pkg.FcklError(st, "fckl_projected_logprobs")
    return logp, entropy, lse


def _projected_backward(dt, N, d, V, T, H, W, tokens, lse, entropy, g_logp, g_entropy, chunk, need, dH=None, dW=None,
                        ws=None, stream=None, round_dW=False):
    """projected_logprobs_backward of checked arguments."""
    import torch
    dev = H.device
    ws = _head_ws(ws, N, d, V, T, chunk, dt, dev, 1)
    if not need[0]:
        dH = None
    elif dH is None:
        dH = torch.empty(N, d, dtype=H.dtype, device=dev)
    if not need[1]:
        dW = None
    elif dW is None:
        dW = torch.empty(V, d, dtype=torch.float32, device=dev)
    dW16 = torch.empty(V, d, dtype=W.dtype, device=dev) if round_dW and dW is not None and dt == _pkg.BF16 else None
    if N == 0 and dW is None:
        return dH, dW
    p = _address
    st = _pkg.load().fckl_projected_logprobs_backward(p(H), p(W), dt, p(tokens), N, d, V, T, chunk, p(lse), p(entropy),
                                                      p(g_logp), p(g_entropy), p(dH), p(dW), p(dW16),
                                                      ws.tensor.data_ptr(), ws.nbytes, _stream(stream))
    if st != _pkg.OK:
        raise _pkg.FcklError(st, "fckl_projected_logprobs_backward")
    return dH, dW if dW16 is None else dW16


def projected_logprobs(H, W, tokens, chunk, ws=None, stream=None):
    """(logp fp32 [N, T], entropy fp32 [N], lse fp32 [N]) of the logits H W^T, ``chunk`` positions
    at a time. ``ws``: Workspace(N, d, V, T, chunk, kind="projected")."""
    shape = _head_args(H, W, tokens)
    _on_device(H.device, H=H, W=W, tokens=tokens)
    with _for_stream(stream, H, W, tokens, ws):
        return _projected(*shape, H, W, tokens, chunk, ws, stream)


def projected_logprobs_backward(H, W, tokens, lse, entropy, g_logp, g_entropy=None, chunk=2048, ws=None, stream=None,
                                dH=None, dW=None, need=(True, True), round_dW=False):
    """(dH [N, d] in H's dtype, dW fp32 [V, d]) of sum g_logp * logp + sum g_entropy * entropy;
    ``lse`` and ``entropy`` as projected_logprobs returned them. ``need``: which of the two to
    compute (the other is None and its product is left out). ``round_dW``: dW in W's dtype instead,
    rounded once from the fp32 sums.
    ``ws``: Workspace(N, d, V, T, chunk, kind="projected_backward")."""
    import torch
    dt, N, d, V, T = _head_args(H, W, tokens)
    dev = H.device
    _on_device(dev, H=H, W=W, tokens=tokens, lse=lse, entropy=entropy, g_logp=g_logp, g_entropy=g_entropy, dH=dH,
               dW=dW)
    f32 = torch.float32
    _dense("lse", lse, f32, (N,))
    _dense("entropy", entropy, f32, (N,))
    _dense("g_logp", g_logp, f32, (N, T))
    if g_entropy is not None:
        _dense("g_entropy", g_entropy, f32, (N,))
    if dH is not None:
        _dense("dH", dH, H.dtype, (N, d))
    if dW is not None:
        _dense("dW", dW, f32, (V, d))
    with _for_stream(stream, H, W, tokens, lse, entropy, g_logp, g_entropy, dH, dW, ws):
        return _projected_backward(dt, N, d, V, T, H, W, tokens, lse, entropy, g_logp, g_entropy, chunk, need, dH, dW,
                                   ws, stream, round_dW)


def _head_autograd_function():
    import torch

    class ProjectedLogprobs(torch.autograd.Function):
        @staticmethod
        def forward(ctx, H, W, tokens, chunk):
            ctx.shape = _head_args(H, W, tokens)
            _on_device(H.device, H=H, W=W, tokens=tokens)
            logp, entropy, lse = _projected(*ctx.shape, H, W, tokens, chunk)
            ctx.save_for_backward(H, W, tokens, lse, entropy)
            ctx.chunk = chunk
            ctx.set_materialize_grads(False)
            return logp, entropy

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, g_logp, g_entropy):
            H, W, tokens, lse, entropy = ctx.saved_tensors
            if g_logp is None and g_entropy is None:
                return None, None, None, None
            ge = None if g_entropy is None else _upstream(g_entropy, None, H.device)
            gl = _upstream(g_logp, tuple(tokens.shape), H.device)
            dH, dW = _projected_backward(*ctx.shape, H, W, tokens, lse, entropy, gl, ge, ctx.chunk,
                                         ctx.needs_input_grad, round_dW=True)
            return dH, dW, None, None

    return ProjectedLogprobs


_ProjectedLogprobs = None


def fused_token_logprobs(H, W, tokens, chunk):
    """(logp [N, T], entropy [N]) of the logits H W^T, differentiable in H and W (W's gradient is
    summed in fp32 and rounded once to W's dtype)."""
    global _ProjectedLogprobs
    if _ProjectedLogprobs is None:
        _ProjectedLogprobs = _head_autograd_function()
    return _ProjectedLogprobs.apply(H, W, tokens, chunk)
