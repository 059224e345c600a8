"""The norm over a set of gradient tensors, and the gradients scaled to at most a given norm.

Argument marshalling only, as in the package itself: every step runs in the CUDA library.

    norm = fckl.gradient_norm([dW, *others])                        # fp32 [1], on the device
    norm = fckl.clip_gradients([p.grad for p in params], 1.0)       # in place
    norm = fckl.clip_gradients(grads, 1.0, out=buckets)             # elsewhere, of another type if wanted

Gradients are bf16, fp16 or fp32, mixed at will, each dense in memory (in any order of its dimensions);
None (a parameter without a gradient) is skipped. Nothing waits for the device.
"""
from __future__ import annotations

import array
import ctypes
import weakref

import chunked_kl_loss_gb300 as _pkg
from .scoring import _for_stream, _here, _stream, _value_code

__all__ = ["gradient_norm", "clip_gradients"]


def _set_argtypes(lib):
    c = ctypes
    vp, i64, i32, sz, f32 = c.c_void_p, c.c_int64, c.c_int, c.c_size_t, c.c_float
    lib.fckl_gradient_norm_workspace_bytes.restype = sz
    lib.fckl_gradient_norm_workspace_bytes.argtypes = [i64]
    lib.fckl_gradient_norm.restype = i32
    lib.fckl_gradient_norm.argtypes = [vp, vp, vp, i32, vp, vp, sz, vp]
    lib.fckl_clip_gradients.restype = i32
    lib.fckl_clip_gradients.argtypes = [vp, vp, vp, i32, f32, vp, vp, vp, vp, sz, vp]


def _dense(t):
    """Whether a tensor's elements fill one stretch of memory, in whatever order of its dimensions."""
    want = 1
    for stride, size in sorted((st, sz) for st, sz in zip(t.stride(), t.shape) if sz != 1):
        if stride != want:
            return False
        want *= size
    return True


def _list(name, tensors, device):
    """(addresses, types, whether all are contiguous) of the tensors, as arrays that the library reads."""
    import torch
    index = -1 if device.type == "cpu" else device.index
    if set(map(torch.Tensor.get_device, tensors)) - {index}:
        where = [t.device for t in tensors if t.get_device() != index]
        raise ValueError(f"{name} must be on one device, got {where[0]} beside {device}")
    contiguous = all(map(torch.Tensor.is_contiguous, tensors))
    if not contiguous:
        for t in tensors:
            if not _dense(t):
                raise ValueError(f"{name} must be dense in memory, got strides {list(t.stride())}")
    codes = {dtype: _value_code(t, name) for dtype, t in {t.dtype: t for t in tensors}.items()}
    if len(codes) == 1:
        types = array.array("i", [*codes.values()]) * len(tensors)
    else:
        types = array.array("i", [codes[t.dtype] for t in tensors])
    return array.array("Q", list(map(torch.Tensor.data_ptr, tensors))), types, contiguous


def _sizes(tensors):
    import torch
    return array.array("q", list(map(torch.Tensor.numel, tensors)))


def _given(tensors):
    """The tensors as a list, without None, and where None stood (None: nowhere)."""
    tensors = list(tensors)
    if type(None) not in set(map(type, tensors)):
        return tensors, None
    return [t for t in tensors if t is not None], [t is None for t in tensors]


def _of(a):
    return a.buffer_info()[0] if len(a) else None


def _device(grads):
    import torch
    index = torch.cuda.current_device()
    device = torch.device("cuda", index)
    if grads and grads[0].device != device:
        raise ValueError(f"tensors must be on the current CUDA device, got {grads[0].device}")
    return device


def _room(count, ws, device):
    import torch
    n = _pkg.load().fckl_gradient_norm_workspace_bytes(count)
    if n == 0:
        raise _pkg.FcklError(_pkg.ERR_UNSUPPORTED, "workspace_bytes")
    if ws is None:
        ws = _pkg._last_ws = _pkg.Workspace.sized(n, device)
    else:
        _pkg._last_ws = weakref.ref(ws)
    return ws, torch.empty(1, dtype=torch.float32, device=device)


def gradient_norm(grads, ws=None, stream=None):
    """The 2-norm over all elements of ``grads``, fp32 [1]. Finite gradients of any size are summed without
    overflow. ``ws``: a Workspace of at least fckl_gradient_norm_workspace_bytes(number of tensors)."""
    grads, _ = _given(grads)
    device = _device(grads)
    ptrs, types, _ = _list("grads", grads, device)
    sizes = _sizes(grads)
    with _for_stream(stream, ws, *grads) if stream is not None else _here:
        ws, norm = _room(len(grads), ws, device)
    st = _pkg.load().fckl_gradient_norm(_of(ptrs), _of(sizes), _of(types), len(grads), norm.data_ptr(),
                                        ws.tensor.data_ptr(), ws.nbytes, _stream(stream))
    if st != _pkg.OK:
        raise _pkg.FcklError(st, "fckl_gradient_norm")
    return norm


def clip_gradients(grads, max_norm, out=None, ws=None, stream=None):
    """Scales ``grads`` by min(1, max_norm / (norm + 1e-6)) and returns the norm before that, fp32 [1]. In
    place, or into ``out``: tensors of the same shapes and memory orders, of any of the three types (the product is
    fp32, rounded once). What is written may overlap no other tensor. A NaN norm makes the gradients NaN, an
    infinite gradient scales the others by 0."""
    import torch
    grads, gaps = _given(grads)
    if out is not None:
        out, out_gaps = _given(out)
        if len(out) != len(grads) or out_gaps != gaps:
            raise ValueError("out must have one tensor for each gradient")
    if not max_norm >= 0:
        raise ValueError(f"max_norm must not be negative, got {max_norm}")
    device = _device(grads)
    ptrs, types, contiguous = _list("grads", grads, device)
    sizes = _sizes(grads)
    to, to_types = ptrs, types
    if out is not None:
        to, to_types, as_well = _list("out", out, device)
        alike = [g.shape for g in grads] == [o.shape for o in out]
        if not alike or not (contiguous and as_well) and any(
                [g.stride() != o.stride() for g, o in zip(grads, out) if not (g.is_contiguous() and o.is_contiguous())]):
            raise ValueError("out must have the gradients' shapes and memory orders")
    with _for_stream(stream, ws, *grads, *(out or ())) if stream is not None else _here:
        ws, norm = _room(len(grads), ws, device)
    st = _pkg.load().fckl_clip_gradients(_of(ptrs), _of(sizes), _of(types), len(grads), float(max_norm), _of(to),
                                         _of(to_types), norm.data_ptr(), ws.tensor.data_ptr(), ws.nbytes,
                                         _stream(stream))
    if st != _pkg.OK:
        raise _pkg.FcklError(st, "fckl_clip_gradients")
    torch.autograd.graph.increment_version(grads if out is None else out)  # a backward pass that saved them raises
    return norm
