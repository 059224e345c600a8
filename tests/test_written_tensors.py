"""Tensors that a caller hands in to be written (out=, dW=, or in place) count as modified for autograd, as
after torch's own in-place operations: a backward pass that would read what was overwritten raises."""
import pytest
import torch

gpu = pytest.mark.gpu


def calls(fckl):
    """name -> (call, the tensors that it writes, the others)."""
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    z, g, out, W, x = r(4, 40), r(4, 40), r(4, 40), r(40, 16), r(6, 16)
    t = torch.tensor([0, 3, 3, -1, 39, 7], dtype=torch.int32, device="cuda")
    h = t[:4].view(4, 1)
    mask = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    a, b = r(300), r(7).bfloat16()
    to = [torch.empty_like(a), torch.empty_like(b)]
    rows, dW = r(6, 16), r(40, 16)
    return {
        "adjust into": (lambda: fckl.adjust_logits(z, h, repetition=2.0, out=out), [out], [z, h]),
        "adjust in place": (lambda: fckl.adjust_logits(z, h, repetition=2.0, out=z), [z], [h]),
        "adjust under a mask": (lambda: fckl.adjust_logits(z, h, repetition=2.0, allowed=mask, out=z), [z], [h, mask]),
        "adjust gradient into": (lambda: fckl.adjust_logits_backward(g, z, h, repetition=2.0, out=out), [out], [g, z, h]),
        "adjust gradient in place": (lambda: fckl.adjust_logits_backward(g, z, h, repetition=2.0, out=g), [g], [z, h]),
        "adjust gradient over the logits": (lambda: fckl.adjust_logits_backward(g, z, h, repetition=2.0, out=z), [z], [g, h]),
        "clip in place": (lambda: fckl.clip_gradients([a, None, b], 0.1), [a, b], []),
        "clip into": (lambda: fckl.clip_gradients([a, b], 0.1, out=to), to, [a, b]),
        "embedding into": (lambda: fckl.embedding(W, t, out=rows), [rows], [W, t]),
        "embedding gradient into": (lambda: fckl.embedding_backward(x, t, 40, dW=dW), [dW], [x, t]),
        "embedding gradient added": (lambda: fckl.embedding_backward(x, t, 40, dW=dW, accumulate=True), [dW], [x, t]),
        "adjust": (lambda: fckl.adjust_logits(z, h, repetition=2.0), [], [z, h]),
        "adjust gradient": (lambda: fckl.adjust_logits_backward(g, z, h, repetition=2.0), [], [g, z, h]),
        "norm": (lambda: fckl.gradient_norm([a, b]), [], [a, b]),
        "embedding": (lambda: fckl.embedding(W, t), [], [W, t]),
        "embedding gradient": (lambda: fckl.embedding_backward(x, t, 40), [], [x, t]),
    }


NAMES = ["adjust into", "adjust in place", "adjust under a mask", "adjust gradient into", "adjust gradient in place",
         "adjust gradient over the logits", "clip in place", "clip into", "embedding into", "embedding gradient into",
         "embedding gradient added", "adjust", "adjust gradient", "norm", "embedding", "embedding gradient"]


@gpu
@pytest.mark.parametrize("name", NAMES)
def test_versions_of_what_is_written(fckl, name):
    call, written, read = calls(fckl)[name]
    before = [t._version for t in written + read]
    call()
    now = [t._version for t in written + read]
    assert fckl.check() == fckl.OK
    k = len(written)
    assert all(n > b for n, b in zip(now[:k], before[:k])) and now[k:] == before[k:]


@gpu
@pytest.mark.parametrize("name", NAMES[:11])
def test_tensors_of_inference_mode_are_taken(fckl, name):
    """They have no version to raise."""
    with torch.inference_mode():
        call, written, _ = calls(fckl)[name]
        call()
    before = [t.clone() for t in written]
    call()
    assert fckl.check() == fckl.OK and all(t.shape == b.shape for t, b in zip(written, before))


@gpu
def test_backward_through_overwritten_tensors_raises(fckl):
    """Logits that the rules' gradient needs, adjusted in place before it is taken; what a torch product
    saved, overwritten by each of the others; a view's base."""
    h = torch.tensor([[3], [5]], dtype=torch.int32, device="cuda")
    leaf = torch.randn(2, 40, device="cuda", requires_grad=True)
    z = leaf * 1.0
    y = fckl.differentiable_adjusted_logits(z, h, repetition=2.0)
    fckl.adjust_logits(z.detach(), h, repetition=2.0, out=z.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    for name, (call, written, _) in calls(fckl).items():
        if not written:
            continue
        w = torch.ones_like(written[0]).requires_grad_()
        y = (w * written[0]).sum()
        call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    base = torch.randn(4, 40, device="cuda")
    w = torch.ones_like(base).requires_grad_()
    y = (w * base).sum()
    fckl.adjust_logits(base[:2], h, repetition=2.0, out=base[:2])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


@gpu
def test_versions_under_capture(fckl):
    """Counted once, when the call is captured."""
    call, (out,), _ = calls(fckl)["adjust in place"]
    call()
    graph, before = torch.cuda.CUDAGraph(), out._version
    with torch.cuda.graph(graph):
        call()
    assert out._version > before
    graph.replay()
    torch.cuda.synchronize()
    assert fckl.check() == fckl.OK
