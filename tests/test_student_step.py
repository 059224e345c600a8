"""The operators around the output matrix used together, as a training step of a student with tied
embeddings uses them: lookup, hidden states, logits under the rules that its answers were sampled by, their
log-probabilities, the KL loss, the gradients of both ends of W in one matrix, and the clipped step."""
import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu
U = 2.0 ** -24


def setting(V=600, d=64, N=90, L=30, seed=0, dtype=torch.float32):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ri = lambda hi, *s: torch.randint(0, hi, s, generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    tokens = ri(V, N)
    tokens[::11] = -1
    keep = torch.rand(N, V, generator=g, device="cuda") < 0.7
    answer = ri(V, N, 1)
    keep.scatter_(1, answer.long(), True)
    pad = torch.nn.functional.pad(keep, (0, -V % 32)).view(N, -1, 32).long()
    bits = (pad << torch.arange(32, device="cuda")).sum(2)
    bits = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).int()
    return dict(W=(r(V, d) / d ** 0.5).to(dtype), mix=r(d, d) / d ** 0.5, tokens=tokens, answer=answer, keep=keep, bits=bits,
                history=ri(V, N, L), lengths=ri(L + 1, N), rep=1 + 0.5 * torch.rand(N, generator=g, device="cuda"),
                g=r(N, 1), ge=0.1 * r(N))


@gpu
def test_policy_term_through_both_ends_of_W(fckl):
    """Gradient of sum g logp + sum ge entropy with respect to W, through the lookup, the output matrix, the
    rules and the softmax, against the same in 64 bits. Each step sums at most V = 600 terms in fp32: a
    relative 600 u of the sums of sizes, which for these sums of random signs are below 4 sqrt(600) times
    the results' largest entry, in four steps: 4 * 600 u * 100 < 0.015; held here to 1e-4, five roundings of
    a sum of 600 terms of random errors (sqrt(600) u * 5 = 7e-6) and a margin of ten."""
    s = setting()
    W = s["W"].clone().requires_grad_()
    x = fckl.differentiable_embedding(W, s["tokens"], scale=8.0)
    z = torch.tanh(x @ s["mix"]) @ W.t()
    y = fckl.differentiable_adjusted_logits(z, s["history"], s["lengths"], repetition=s["rep"], allowed=s["bits"])
    logp, entropy = fckl.differentiable_token_logprobs(y, s["answer"])
    dW, = torch.autograd.grad((logp, entropy), W, (s["g"], s["ge"]))
    assert fckl.check() == fckl.OK

    W64 = s["W"].double().requires_grad_()
    e = torch.where(s["tokens"][:, None] < 0, 0.0, 8.0 * W64[s["tokens"].clamp(min=0).long()])
    z64 = torch.tanh(e @ s["mix"].double()) @ W64.t()
    N, V = z64.shape
    live = torch.arange(s["history"].shape[1], device="cuda") < s["lengths"][:, None]
    seen = torch.zeros(N, V + 1, dtype=torch.bool, device="cuda")
    seen.scatter_(1, torch.where(live, s["history"], V).long(), True)
    rep = s["rep"].double()[:, None]
    y64 = torch.where(seen[:, :V], torch.where(z64 > 0, z64 / rep, z64 * rep), z64)
    lq = torch.log_softmax(y64.masked_fill(~s["keep"], -float("inf")), 1)
    q = lq.exp()
    ent = -(q * lq.masked_fill(~s["keep"], 0.0)).sum(1)
    at = lq.gather(1, s["answer"].long())
    want, = torch.autograd.grad((at, ent), W64, (s["g"].double(), s["ge"].double()))
    assert (logp.double() - at).abs().max() <= 1e-4 and (entropy.double() - ent).abs().max() <= 1e-4
    assert (dW.double() - want).abs().max() <= 1e-4 * want.abs().max()


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tied_step(fckl, dtype):
    """The loss's dW, the lookup's gradient added to it, and both clipped with the others: the sum is the
    two gradients' own, rounded once, and after clipping the norm is the wanted one."""
    s = setting(dtype=dtype)
    N, V = 90, 600
    idx = torch.argsort(torch.rand(N, V, device="cuda"), 1)[:, :20].int().contiguous()
    logp = torch.log_softmax(torch.randn(N, 20, device="cuda"), 1) - 0.1
    H = fckl.embedding(s["W"], s["tokens"], scale=8.0)
    loss, lse, dH, dW = fckl.forward_backward(H, s["W"], idx, logp, 32, grad_scale=1 / N)
    fckl.check()
    alone = fckl.embedding_backward(dH, s["tokens"], V, scale=8.0)
    both = fckl.embedding_backward(dH, s["tokens"], V, scale=8.0, dW=dW.clone(), accumulate=True)
    size = alone.abs() + dW.abs()
    assert ((both.double() - alone.double() - dW.double()).abs() <= 2 * U * size).all()
    others = [dH, torch.randn(7, device="cuda").bfloat16()]
    before = [t.clone() for t in (both, *others)]
    norm = fckl.clip_gradients([both, *others], 0.05)
    want = np.sqrt(sum(float(t.double().square().sum()) for t in before))
    assert abs(float(norm) - want) <= 17 * U * want
    assert want > 0.05
    # the largest share of the norm lies in fp32 and bf16 values that are each off by half a step
    after = fckl.gradient_norm([both, *others])
    assert abs(float(after) - 0.05) <= 0.05 * (2.0 ** -8 + 1e-5)


@gpu
def test_captured_scoring_step(fckl):
    """Rules, scores and their gradient captured once and replayed on new logits."""
    s = setting()
    z = torch.randn(90, 600, device="cuda")
    k = dict(repetition=s["rep"], allowed=s["bits"])

    def step():
        y = fckl.adjust_logits(z, s["history"], s["lengths"], **k)
        logp, entropy, norm, _, _ = fckl.token_logprobs(y, s["answer"])
        dy = fckl.token_logprobs_backward(y, s["answer"], norm, entropy, s["g"], s["ge"])
        dz = fckl.adjust_logits_backward(dy, z, s["history"], s["lengths"], out=dy, **k)
        return logp, dz, fckl.clip_gradients([dz], 1.0)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    z.copy_(torch.randn(90, 600, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))
