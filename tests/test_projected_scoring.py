"""Scoring from hidden states (projected_logprobs and its gradients) against the fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24):
* bf16 products are exact in fp32; a logit is a sum of d of them accumulated in fp32 in some order,
  each addition truncated at worst (a whole step, 2u) of the running sum: |dz| <= 2 d u sum |h w|, and
  sum |h w| <= |h| |w| (norms). The statistics add r (a tile's 256 values and the tiles' merges), as
  for logits at hand. For fp32 inputs the oracle gets the tf32-rounded inputs, whose products are
  exact in fp32 as well.
* G is rounded to bf16 (half a step, 2^-8 relative) and dH, dW sum V and N such entries: off by at
  most 2^-8 sum |G| |w| (resp. |h|), plus the products' own sums and the rounding of dH to its type.
  For fp32 inputs the factor w (h) is rounded to bf16 too: twice 2^-8.
"""
import ctypes

import numpy as np
import pytest
import torch

import synthetic
from oracle import scoring_oracle as orc

gpu = pytest.mark.gpu
U = 2.0 ** -24


def make(N, d, V, T, dtype, seed, sharp=1.0):
    rng = np.random.default_rng(seed)
    H = (rng.normal(size=(N, d)) * sharp).astype(np.float32)
    W = (rng.normal(size=(V, d)) / np.sqrt(d)).astype(np.float32)
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    Ht, Wt = torch.from_numpy(H).cuda().to(tdt), torch.from_numpy(W).cuda().to(tdt)
    tokens = rng.integers(0, V, size=(N, T))
    tokens[rng.random((N, T)) < 0.1] = -1
    if T > 2:
        tokens[:, 1] = tokens[:, 0]  # repeats
    return Ht, Wt, torch.from_numpy(tokens).int().cuda()


def exact_inputs(Ht, Wt):
    H, W = Ht.float().cpu().numpy(), Wt.float().cpu().numpy()
    if Ht.dtype == torch.float32:
        H, W = synthetic.round_tf32(H), synthetic.round_tf32(W)
    return H.astype(np.float64), W.astype(np.float64)


def close(got, want, tol):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], np.broadcast_to(tol, got.shape)[bad][:4])


def f64(t):
    return t.detach().cpu().double().numpy()


def logit_error(H, W):
    """Per position, the most that a logit can be off."""
    return 2 * H.shape[1] * U * np.linalg.norm(H, axis=1) * np.linalg.norm(W, axis=1).max() + 4 * U


def check(fckl, Ht, Wt, tokens, chunk, with_entropy=True, seed=0):
    logp, ent, lse = fckl.projected_logprobs(Ht, Wt, tokens, chunk)
    assert fckl.check() == fckl.OK
    H, W = exact_inputs(Ht, Wt)
    tk = tokens.cpu().numpy()
    w_logp, w_ent, w_lse = orc.projected(H, W, tk)
    V, r = W.shape[0], (256 + W.shape[0] // 8192 + 80) * U + 2.0 ** -21
    dz = logit_error(H, W)
    close(f64(lse), w_lse, dz + r + 8 * U * np.abs(w_lse))
    close(f64(logp), w_logp, (2 * dz + r)[:, None] + 8 * U * np.abs(w_logp))
    spread = np.maximum(w_ent, np.log(V)) + 2
    close(f64(ent), w_ent, (dz * 2 * spread + r * (1 + 2 * spread)))

    rng = np.random.default_rng(seed)
    g = rng.normal(size=tk.shape).astype(np.float32)
    ge = rng.normal(size=len(H)).astype(np.float32) if with_entropy else np.zeros(len(H), np.float32)
    dH, dW = fckl.projected_logprobs_backward(Ht, Wt, tokens, lse, ent, torch.from_numpy(g).cuda(),
                                              torch.from_numpy(ge).cuda() if with_entropy else None, chunk=chunk)
    assert fckl.check() == fckl.OK
    G = orc.logits_gradient(H @ W.T, tk, g, ge)
    w_dH, w_dW = G @ W, G.T @ H
    half = 2.0 ** -8 * (2 if Ht.dtype == torch.float32 else 1)
    # G's own error before its rounding: q off by its exponent's, factors of the upstream sums
    lq = orc._log_softmax(H @ W.T)[0]
    q = np.exp(lq)
    a = np.abs(np.where(tk < 0, 0, g)).sum(1, keepdims=True) + np.abs(ge)[:, None] * (1 + np.abs(lq) + w_ent[:, None])
    eG = half * 1.01 * np.abs(G) + q * a * (4 * (dz + r)[:, None] * (1 + spread[:, None]) + 2.0 ** -19)
    out = 2.0 ** -8 if Ht.dtype == torch.bfloat16 else 2.0 ** -23
    close(f64(dH), w_dH, eG @ np.abs(W) + 4 * V * U * (np.abs(G) @ np.abs(W)) / 16 + out * np.abs(w_dH) + 1e-30)
    close(f64(dW), w_dW, eG.T @ np.abs(H) + 4 * len(H) * U * (np.abs(G).T @ np.abs(H)) + 1e-30)
    return logp, ent, lse, dH, dW


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,d,V,T,chunk", [
    (1, 8, 1, 1, 1), (1, 64, 300, 1, 16), (5, 72, 257, 3, 2), (130, 256, 2057, 2, 100), (256, 128, 256, 1, 256),
    (300, 320, 1000, 20, 128), (33, 1024, 5001, 4, 2048), (2, 2880, 700, 300, 8), (520, 64, 4100, 1, 512),
])
def test_projected(fckl, dtype, N, d, V, T, chunk):
    check(fckl, *make(N, d, V, T, dtype, seed=N + V), chunk)


@gpu
@pytest.mark.parametrize("N,d,V,T", [
    (1, 2880, 5000, 1), (2, 8, 1, 1), (7, 64, 200, 3), (8, 520, 1000, 32), (9, 128, 333, 2), (24, 256, 4097, 1),
    (25, 72, 17, 4), (32, 1000, 16, 1), (32, 2880, 3000, 2), (16, 4096, 700, 0), (32, 4096, 700, 1), (33, 512, 900, 1),
    (3, 256, 900, 33), (1, 2880, 100003, 1),
])
def test_projected_decode(fckl, N, d, V, T):
    """Few positions: both sides of every limit of the decoding form (positions, tokens, shared
    memory), odd vocabularies, a vocabulary below one step."""
    Ht, Wt, tokens = make(N, d, V, max(T, 1), "bf16", seed=N + V)
    tokens = tokens[:, :T].contiguous()
    logp, ent, lse = fckl.projected_logprobs(Ht, Wt, tokens, 2048)
    assert fckl.check() == fckl.OK
    H, W = exact_inputs(Ht, Wt)
    w_logp, w_ent, w_lse = orc.projected(H, W, tokens.cpu().numpy())
    dz, r = logit_error(H, W), (V // 16 + 80) * U + 2.0 ** -21
    close(f64(lse), w_lse, dz + r + 8 * U * np.abs(w_lse))
    close(f64(logp), w_logp, (2 * dz + r)[:, None] + 8 * U * np.abs(w_logp))
    spread = np.maximum(w_ent, np.log(V)) + 2
    close(f64(ent), w_ent, (dz * 2 * spread + r * (1 + 2 * spread)))
    again = fckl.projected_logprobs(Ht, Wt, tokens, 2048)
    assert all(torch.equal(a, b) for a, b in zip(again, (logp, ent, lse)))


@gpu
def test_projected_decode_bad_token(fckl):
    Ht, Wt, tokens = make(2, 64, 500, 2, "bf16", 2)
    tokens[0, 1] = 500
    logp = fckl.projected_logprobs(Ht, Wt, tokens, 4)[0]
    assert fckl.check(raise_on_error=False) == fckl.ERR_INDEX
    assert torch.isnan(logp[0, 1]) and torch.isfinite(logp[1]).all()


@gpu
def test_projected_without_tokens_and_without_entropy(fckl):
    Ht, Wt, tokens = make(40, 128, 900, 2, "bf16", 3)
    check(fckl, Ht, Wt, tokens, 16, with_entropy=False)
    check(fckl, Ht, Wt, tokens[:, :0].contiguous(), 16)
    # every slot empty
    none = torch.full_like(tokens, -1)
    logp, ent, lse, dH, dW = check(fckl, Ht, Wt, none, 16, with_entropy=False)
    assert (logp == 0).all() and (dH == 0).all() and (dW == 0).all()


@gpu
def test_projected_sharp(fckl):
    """Logits of tens: the softmax is all but one-hot, its entropy near 0."""
    check(fckl, *make(64, 256, 3000, 2, "bf16", 9, sharp=12.0), 64)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("level", [-200.0, 200.0])
def test_projected_far_from_zero(fckl, dtype, level):
    """Every logit near -200 or 200: a place past the vocabulary (logit 0 in the last tile) may not
    count, nor its exponential, inf, reach a product."""
    Ht, Wt, tokens = make(40, 64, 1001, 2, dtype, 11, sharp=0.01)
    check(fckl, Ht + level / 64, Wt * 0.125 + 1.0, tokens, 16)


@gpu
def test_projected_large_vocabulary(fckl):
    """The vocabulary of the workloads, a decode-sized batch; forward only."""
    Ht, Wt, tokens = make(3, 256, 201088, 2, "bf16", 4)
    logp, ent, lse = fckl.projected_logprobs(Ht, Wt, tokens, 2048)
    H, W = exact_inputs(Ht, Wt)
    w_logp, w_ent, w_lse = orc.projected(H, W, tokens.cpu().numpy())
    tol = 2 * logit_error(H, W) + 400 * U + 2.0 ** -21
    close(f64(lse), w_lse, tol)
    close(f64(logp), w_logp, tol[:, None] + 8 * U * np.abs(w_logp))
    close(f64(ent), w_ent, 30 * tol)


@gpu
def test_projected_matches_loss_statistics(fckl):
    """The loss against a one-token teacher of mass 1 is minus the log-probability: same lse, same
    gradient, to the loss's tolerances."""
    N, d, V = 200, 256, 3001
    Ht, Wt, tokens = make(N, d, V, 1, "bf16", 6)
    tokens = tokens.clamp(min=0)
    logp, ent, lse = fckl.projected_logprobs(Ht, Wt, tokens, 64)
    zero = torch.zeros(N, 1, device="cuda")
    loss, lse2, dH2, dW2 = fckl.forward_backward(Ht, Wt, tokens, zero, 64)
    fckl.check()
    assert torch.allclose(lse, lse2, atol=1e-4)
    assert abs(float(loss) + float(logp.sum())) <= 1e-4 * abs(float(loss))
    dH, dW = fckl.projected_logprobs_backward(Ht, Wt, tokens, lse, ent, -torch.ones(N, 1, device="cuda"), chunk=64)
    fckl.check()
    assert (dH.float() - dH2.float()).abs().max() <= 2e-2 * dH2.float().abs().max()
    assert (dW - dW2).abs().max() <= 2e-2 * dW2.abs().max()


@gpu
def test_projected_autograd(fckl):
    """Gradients through autograd: the direct call's, W's rounded to its type; a missing and a
    broadcast upstream gradient; only one leaf wanting a gradient; differences of the oracle."""
    Ht, Wt, tokens = make(50, 128, 700, 2, "bf16", 8)
    H, W = Ht.clone().requires_grad_(), Wt.clone().requires_grad_()
    logp, ent = fckl.fused_token_logprobs(H, W, tokens, 32)
    (logp.sum() - 0.25 * ent.sum()).backward()
    _, ent0, lse0 = fckl.projected_logprobs(Ht, Wt, tokens, 32)
    one = torch.ones(50, 2, device="cuda")
    dH, dW = fckl.projected_logprobs_backward(Ht, Wt, tokens, lse0, ent0, one, torch.full((50,), -0.25, device="cuda"),
                                              chunk=32)
    assert torch.equal(H.grad, dH) and torch.equal(W.grad, dW.to(torch.bfloat16))
    W2 = Wt.clone().requires_grad_()
    fckl.fused_token_logprobs(Ht, W2, tokens, 32)[1].mean().backward()  # entropy alone
    zero = torch.zeros(50, 2, device="cuda")
    _, dW = fckl.projected_logprobs_backward(Ht, Wt, tokens, lse0, ent0, zero, torch.full((50,), 1 / 50, device="cuda"),
                                             chunk=32)
    assert torch.equal(W2.grad, dW.to(torch.bfloat16))
    # directional differences of the fp64 value; bf16 gradients: each entry within 2^-7 of itself
    # and G's rounding, so the sum over random directions within 2^-6 of its root sum of squares
    Hd, Wd = exact_inputs(Ht, Wt)
    tk = tokens.cpu().numpy()
    value = lambda h, w: (lambda a, b, _: a.sum() - 0.25 * b.sum())(*orc.projected(h, w, tk))  # noqa: E731
    rng = np.random.default_rng(1)
    for A, grad, f in ((Hd, f64(H.grad), lambda x: value(x, Wd)), (Wd, f64(W.grad), lambda x: value(Hd, x))):
        for _ in range(3):
            v = rng.normal(size=A.shape)
            diff = (f(A + 1e-5 * v) - f(A - 1e-5 * v)) / 2e-5
            assert abs(diff - (grad * v).sum()) <= 2.0 ** -6 * np.sqrt(((grad * v) ** 2).sum()) + 1e-6 * abs(diff)


@gpu
@pytest.mark.parametrize("N,T,chunk,same", [(1, 1, 1, False), (40, 1, 16, False), (300, 2, 128, True), (64, 3, 64, False),
                                            (90, 8, 40, True), (700, 1, 512, True)])
def test_projected_token_entries_keep_precision(fckl, N, T, chunk, same):
    """Up to 8 tokens: only the dense part of G carries bf16 rounding, not its entries at the tokens
    (repeated ones, and one token for most positions, among them). dW is compared as fp32; dH's own
    rounding is bf16's."""
    d, V = 192, 1500
    Ht, Wt, tokens = make(N, d, V, T, "bf16", seed=N + T)
    if same:
        tokens[::2] = 77
    _, ent, lse = fckl.projected_logprobs(Ht, Wt, tokens, chunk)
    g = torch.randn(N, T, device="cuda")
    dH, dW = fckl.projected_logprobs_backward(Ht, Wt, tokens, lse, ent, g, chunk=chunk)
    assert fckl.check() == fckl.OK
    H, W = exact_inputs(Ht, Wt)
    tk, gn = tokens.cpu().numpy(), f64(g)
    gn = np.where(tk < 0, 0, gn)
    G = orc.logits_gradient(H @ W.T, tk, gn)
    q = np.exp(orc._log_softmax(H @ W.T)[0])
    a = np.abs(gn).sum(1, keepdims=True)
    dz, r = logit_error(H, W)[:, None], (256 + 92) * U + 2.0 ** -21
    eG = q * a * (2.0 ** -8 * 1.01 + 4 * (dz + r) + 2.0 ** -19) + 8 * U * np.abs(G)
    sums = 4 * max(N, V // 16) * U
    close(f64(dW), G.T @ H, eG.T @ np.abs(H) + sums * (np.abs(G).T @ np.abs(H)) + 1e-30)
    want = G @ W
    close(f64(dH), want, eG @ np.abs(W) + sums * (np.abs(G) @ np.abs(W)) + 2.0 ** -8 * np.abs(want) + 1e-30)
    again = fckl.projected_logprobs_backward(Ht, Wt, tokens, lse, ent, g, chunk=chunk)
    assert torch.equal(again[0], dH) and torch.equal(again[1], dW)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_projected_one_gradient(fckl, dtype):
    """A frozen output matrix, or fixed hidden states: the other gradient has the same bits."""
    Ht, Wt, tokens = make(70, 128, 900, 2, dtype, 14)
    _, ent, lse = fckl.projected_logprobs(Ht, Wt, tokens, 32)
    g = torch.randn(70, 2, device="cuda")
    dH, dW = fckl.projected_logprobs_backward(Ht, Wt, tokens, lse, ent, g, chunk=32)
    a, none = fckl.projected_logprobs_backward(Ht, Wt, tokens, lse, ent, g, chunk=32, need=(True, False))
    assert none is None and torch.equal(a, dH)
    none, b = fckl.projected_logprobs_backward(Ht, Wt, tokens, lse, ent, g, chunk=32, need=(False, True))
    assert none is None and torch.equal(b, dW)
    H = Ht.clone().requires_grad_()
    (fckl.fused_token_logprobs(H, Wt, tokens, 32)[0] * g).sum().backward()
    assert torch.equal(H.grad, dH)
    for need in ((True, True), (False, True)):
        c, e = fckl.projected_logprobs_backward(Ht, Wt, tokens, lse, ent, g, chunk=32, need=need, round_dW=True)
        assert torch.equal(e, dW.to(Wt.dtype)) and (c is None or torch.equal(c, dH))
    none, e = fckl.projected_logprobs_backward(Ht[:0], Wt, tokens[:0], lse[:0], ent[:0], g[:0], chunk=32, round_dW=True)
    assert e.dtype == Wt.dtype and (e == 0).all()


@gpu
def test_projected_deterministic_streams_graph_and_chunks(fckl):
    Ht, Wt, tokens = make(300, 256, 5000, 3, "bf16", 10)
    g, ge = torch.randn(300, 3, device="cuda"), torch.randn(300, device="cuda")
    a = fckl.projected_logprobs(Ht, Wt, tokens, 100)
    da = fckl.projected_logprobs_backward(Ht, Wt, tokens, a[2], a[1], g, ge, chunk=100)
    b = fckl.projected_logprobs(Ht, Wt, tokens, 300)
    assert all(torch.equal(x, y) for x, y in zip(a, b))  # the chunk does not change a position's result
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    c = fckl.projected_logprobs(Ht, Wt, tokens, 100, stream=side)
    dc = fckl.projected_logprobs_backward(Ht, Wt, tokens, c[2], c[1], g, ge, chunk=100, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a + da, c + dc))
    ws = fckl.Workspace(300, 256, 5000, 3, 100, kind="projected_backward")
    wf = fckl.Workspace(300, 256, 5000, 3, 100, kind="projected")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e = fckl.projected_logprobs(Ht, Wt, tokens, 100, ws=wf)
        de = fckl.projected_logprobs_backward(Ht, Wt, tokens, e[2], e[1], g, ge, chunk=100, ws=ws)
        dr = fckl.projected_logprobs_backward(Ht, Wt, tokens, e[2], e[1], g, ge, chunk=100, ws=ws, round_dW=True)
    graph.replay()
    torch.cuda.synchronize()
    assert fckl.check(ws) == fckl.OK and fckl.check(wf) == fckl.OK
    assert all(torch.equal(x, y) for x, y in zip(a + da, e + de))
    assert torch.equal(dr[0], da[0]) and torch.equal(dr[1], da[1].to(Wt.dtype))


@gpu
def test_projected_bad_token_and_empty(fckl):
    Ht, Wt, tokens = make(4, 64, 500, 2, "bf16", 2)
    bad = tokens.clone()
    bad[1, 0] = 500
    ws = fckl.Workspace(4, 64, 500, 2, 4, kind="projected")
    logp = fckl.projected_logprobs(Ht, Wt, bad, 4, ws=ws)[0]
    assert fckl.check(ws, raise_on_error=False) == fckl.ERR_INDEX
    assert torch.isnan(logp[1, 0]) and torch.isfinite(logp[0]).all()
    logp, ent, lse = fckl.projected_logprobs(Ht[:0], Wt, tokens[:0], 4)
    assert fckl.check() == fckl.OK and tuple(logp.shape) == (0, 2) and tuple(ent.shape) == (0,)
    dW = torch.full((500, 64), 7.0, device="cuda")
    dH, dW = fckl.projected_logprobs_backward(Ht[:0], Wt, tokens[:0], lse, ent, logp, chunk=4, dW=dW)
    assert tuple(dH.shape) == (0, 64) and (dW == 0).all()


# ------------------------------------------------------------------ refusals and sizes (CPU)
def test_argument_errors_launch_nothing(fckl):
    lib = fckl.load()
    before = lib.fckl_launch_count()
    p, z, odd = ctypes.c_void_p(256), ctypes.c_void_p(0), ctypes.c_void_p(258)
    big = 1 << 40

    def fwd(H=p, W=p, dt=0, tok=p, N=64, d=256, V=4096, T=2, chunk=16, logp=p, ent=p, lse=p, ws=p, n=big):
        return lib.fckl_projected_logprobs(H, W, dt, tok, N, d, V, T, chunk, logp, ent, lse, ws, n, z)

    for bad in (dict(N=-1), dict(T=-1), dict(V=0), dict(d=0), dict(chunk=0), dict(dt=2), dict(H=z), dict(H=odd),
                dict(W=z), dict(W=odd), dict(tok=z), dict(tok=ctypes.c_void_p(257)), dict(logp=z), dict(ent=z),
                dict(lse=z), dict(lse=odd), dict(ws=z), dict(ws=ctypes.c_void_p(128))):
        assert fwd(**bad) == fckl.ERR_ARG, bad
    for bad in (dict(T=1025), dict(d=250), dict(V=(1 << 30) + 1), dict(N=1 << 30, chunk=(1 << 24) + 1)):
        assert fwd(**bad) == fckl.ERR_UNSUPPORTED, bad
    assert fwd(n=256) == fckl.ERR_WORKSPACE

    def bwd(H=p, W=p, dt=0, tok=p, N=64, d=256, V=4096, T=2, chunk=16, lse=p, ent=p, g=p, ge=z, dH=p, dW=p, dW16=z,
            ws=p, n=big):
        return lib.fckl_projected_logprobs_backward(H, W, dt, tok, N, d, V, T, chunk, lse, ent, g, ge, dH, dW, dW16, ws,
                                                    n, z)

    for bad in (dict(lse=z), dict(ent=z), dict(g=z), dict(dH=z, dW=z), dict(dW=odd), dict(dH=odd),
                dict(dW=z, dW16=p), dict(dW16=odd),
                dict(ge=ctypes.c_void_p(257))):
        assert bwd(**bad) == fckl.ERR_ARG, bad
    assert bwd(n=256) == fckl.ERR_WORKSPACE
    assert lib.fckl_launch_count() == before


def test_workspace_sizes(fckl):
    n = fckl.load().fckl_projected_logprobs_workspace_bytes
    f = n(32768, 2880, 201088, 1, 2048, fckl.BF16, 0)
    b = n(32768, 2880, 201088, 1, 2048, fckl.BF16, 1)
    tiles = -(-201088 // 128)
    assert 0 <= f - (3 * tiles * 2048 * 4 + 2 * 2048 * 4) < 8 * 1024 + 32 * 2880 * 2  # statistics, not logits
    # one chunk's gradient slab, 4 to 16 partial dH of a chunk, the ordered tokens
    b -= 2048 * 201088 * 2 + 4 * 2048 * 4
    assert 4 * 2048 * 2880 * 4 <= b < 16 * 2048 * 2880 * 4 + 8 * 1024 + 32 * 2880 * 2
    assert f == n(65536, 2880, 201088, 1, 2048, fckl.BF16, 0)  # the chunk bounds it, not N
    assert n(0, 2880, 201088, 0, 2048, fckl.BF16, 0) > 0
    for bad in ((-1, 64, 100, 1, 16, 0, 0), (4, 60, 100, 1, 16, 0, 0), (4, 64, 100, 1025, 16, 0, 0),
                (4, 64, 100, 1, 0, 0, 0), (4, 64, 100, 1, 16, 2, 0)):
        assert n(*bad) == 0, bad


@pytest.mark.parametrize("bad", [
    lambda f, H, W, t: f.projected_logprobs(H, W, t, 4), lambda f, H, W, t: f.projected_logprobs(H, W.float(), t, 4),
    lambda f, H, W, t: f.projected_logprobs(H.half(), W.half(), t, 4),
    lambda f, H, W, t: f.projected_logprobs(H, W, t.long(), 4),
    lambda f, H, W, t: f.projected_logprobs(H, W[:, :8], t, 4), lambda f, H, W, t: f.projected_logprobs(H[0], W, t, 4),
    lambda f, H, W, t: f.fused_token_logprobs(H, W, t[:2], 4),
    lambda f, H, W, t: f.projected_logprobs_backward(H, W, t, t, t, t),
])
def test_binding_refusals(fckl, bad):
    H, W = torch.zeros(3, 16, dtype=torch.bfloat16), torch.zeros(50, 16, dtype=torch.bfloat16)
    with pytest.raises((TypeError, ValueError)):
        bad(fckl, H, W, torch.zeros(3, 2, dtype=torch.int32))


@gpu
@pytest.mark.parametrize("T", [1, 3])
def test_projected_gradient_without_entropy_does_not_read_it(fckl, T):
    """Where no gradient comes in through the entropy, what stands in its place does not matter."""
    Ht, Wt, tokens = make(70, 128, 900, T, "bf16", 15)
    _, ent, lse = fckl.projected_logprobs(Ht, Wt, tokens, 32)
    g = torch.randn(70, T, device="cuda")
    want = fckl.projected_logprobs_backward(Ht, Wt, tokens, lse, ent, g, chunk=32)
    nothing = torch.full_like(ent, float("nan"))
    assert torch.isfinite(want[1]).all()
    for ge in (None, torch.zeros(70, device="cuda")):
        got = fckl.projected_logprobs_backward(Ht, Wt, tokens, lse, nothing, g, ge, chunk=32)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ logits of any finite size
@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [5, 40, 600])
@pytest.mark.parametrize("kind", ["one far up", "up and down"])
def test_projected_finite_logits_of_any_size(fckl, dtype, N, kind):
    """One logit of 3e38, and with it one of -3e38, beside ordinary ones: each logit has one product that
    is not zero, so that it is exact in fp32. q is 1 at that token and 0 elsewhere; the entropy is 0, and
    the gradient is G = g at the position's token, -g at token 0 (each within bf16's half a step)."""
    d, V = 64, 1001
    rng = np.random.default_rng(N)
    H, W = np.zeros((N, d), np.float32), np.zeros((V, d), np.float32)
    H[:, 0] = 2.0 ** 64
    W[2:, 0] = rng.choice([-2.0, -0.5, 0.25, 1.0, 3.0], V - 2) * 2.0 ** -64
    W[0, 0] = 1.75 * 2.0 ** 63                                       # 2.98e38
    W[1, 0] = -1.75 * 2.0 ** 63 if kind == "up and down" else 2.0 ** -64
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    Ht, Wt = torch.from_numpy(H).cuda().to(tdt), torch.from_numpy(W).cuda().to(tdt)
    tk = rng.integers(2, V, size=(N, 1))
    tk[::2] = 0
    tokens = torch.from_numpy(tk).int().cuda()
    logp, ent, lse = fckl.projected_logprobs(Ht, Wt, tokens, 512)
    assert fckl.check() == fckl.OK
    assert (ent == 0).all() and (lse == 1.75 * 2.0 ** 127).all()
    want = np.where(tk == 0, 0.0, -1.75 * 2.0 ** 127)
    close(f64(logp), want, 2 * U * np.abs(want))
    g = rng.normal(size=(N, 1)).astype(np.float32)
    gt = torch.from_numpy(g).cuda()
    for ge in (None, torch.randn(N, device="cuda")):
        dH, dW = fckl.projected_logprobs_backward(Ht, Wt, tokens, lse, ent, gt, ge, chunk=512)
        assert fckl.check() == fckl.OK
        G = np.zeros((N, V))
        np.put_along_axis(G, tk, np.where(tk == 0, 0.0, g.astype(np.float64)), 1)
        G[:, 0] = np.where(tk[:, 0] == 0, 0.0, -g[:, 0].astype(np.float64))
        w_dH, w_dW = G @ W.astype(np.float64), G.T @ H.astype(np.float64)
        close(f64(dH), w_dH, 2.0 ** -7 * (np.abs(G) @ np.abs(W)) * 1.01)
        close(f64(dW), w_dW, 2.0 ** -8 * (np.abs(G).T @ np.abs(H)) * 1.01 + 4 * N * U * (np.abs(G).T @ np.abs(H)))


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [3, 33])
def test_projected_all_logits_far_down(fckl, dtype, N):
    """Every logit -2.98e38, equal ones: the places past the vocabulary in the last tile do not count."""
    d, V = 64, 1001
    H, W = torch.zeros(N, d), torch.zeros(V, d)
    H[:, 0], W[:, 0] = -(2.0 ** 64), 1.75 * 2.0 ** 63
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    tokens = torch.arange(N, dtype=torch.int32).view(N, 1).cuda() * 30
    logp, ent, lse = fckl.projected_logprobs(H.cuda().to(tdt), W.cuda().to(tdt), tokens, 64)
    assert fckl.check() == fckl.OK
    r = (256 + 92) * U + 2.0 ** -21
    assert (lse == -1.75 * 2.0 ** 127).all()
    close(f64(logp), np.full((N, 1), -np.log(V)), r + 8 * U * np.log(V))
    close(f64(ent), np.full(N, np.log(V)), r * (1 + 2 * np.log(V)))


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_projected_chunk_does_not_change_a_position(fckl, dtype):
    """Chunks on both sides of the sizes at which the statistics' merge takes another block shape, and a
    short last chunk: the same bits."""
    Ht, Wt, tokens = make(1300, 64, 20011, 2, dtype, 12)
    want = fckl.projected_logprobs(Ht, Wt, tokens, 1300)
    assert fckl.check() == fckl.OK
    for chunk in (100, 512, 513, 600, 1299):
        got = fckl.projected_logprobs(Ht, Wt, tokens, chunk)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), chunk


# ------------------------------------------------------------------ dW rounded on the second stream
def _round_both(fckl, monkeypatch, args, ge, chunk, **kw):
    """dH, bf16 dW with the rounding beside the last dH product and after it."""
    out = []
    for how in ("1", "0"):
        monkeypatch.setenv("FCKL_OVERLAP", how)
        out.append(fckl.projected_logprobs_backward(*args, ge, chunk=chunk, round_dW=True, **kw))
        assert fckl.check() == fckl.OK
    return out


@gpu
@pytest.mark.parametrize("N,d,V,T,chunk", [
    (300, 256, 5000, 1, 300), (300, 256, 5000, 3, 100), (301, 128, 3001, 8, 100), (301, 128, 3001, 9, 150),
    (257, 64, 1000, 2, 256), (40, 8, 300, 0, 7), (1100, 512, 8192, 1, 1024),
])
def test_projected_dW_rounded_beside_dH(fckl, monkeypatch, N, d, V, T, chunk):
    """The fork to the second stream and the join: the bits of the rounding in order, with one and several
    chunks, a last chunk of few rows, tokens on both sides of the limit of their kept rests, on another
    stream. dW is overwritten on the caller's stream right behind the call: were it not joined, the
    rounding could read that."""
    Ht, Wt, tokens = make(N, d, V, max(T, 1), "bf16", seed=N + V)
    tokens = tokens[:, :T].contiguous()
    _, ent, lse = fckl.projected_logprobs(Ht, Wt, tokens, chunk)
    g, ge = torch.randn(N, T, device="cuda"), torch.randn(N, device="cuda")
    args = (Ht, Wt, tokens, lse, ent, g)
    dH, dW = fckl.projected_logprobs_backward(*args, ge, chunk=chunk)
    (a, ra), (b, rb) = _round_both(fckl, monkeypatch, args, ge, chunk)
    assert torch.equal(a, dH) and torch.equal(b, dH) and torch.equal(ra, rb) and torch.equal(ra, dW.to(Wt.dtype))
    monkeypatch.setenv("FCKL_OVERLAP", "1")
    torch.cuda.synchronize()
    for stream in (None, torch.cuda.Stream()):
        for _ in range(5):
            scratch = torch.zeros(V, d, device="cuda")
            torch.cuda.synchronize()
            c, rc = fckl.projected_logprobs_backward(*args, ge, chunk=chunk, round_dW=True, dW=scratch, stream=stream)
            with torch.cuda.stream(stream or torch.cuda.current_stream()):
                scratch.fill_(float("nan"))
            torch.cuda.synchronize()
            assert torch.equal(c, dH) and torch.equal(rc, ra)


@gpu
def test_projected_dW_rounded_beside_dH_in_a_graph(fckl, monkeypatch):
    """Captured: the second stream joins the capture and leaves it with the call; replays on new inputs
    give the eager call's bits."""
    monkeypatch.setenv("FCKL_OVERLAP", "1")
    N, d, V, T, chunk = 300, 256, 5000, 2, 128
    Ht, Wt, tokens = make(N, d, V, T, "bf16", 21)
    g = torch.randn(N, T, device="cuda")
    _, ent, lse = fckl.projected_logprobs(Ht, Wt, tokens, chunk)
    args = (Ht, Wt, tokens, lse, ent, g)
    want = fckl.projected_logprobs_backward(*args, chunk=chunk, round_dW=True)
    ws = fckl.Workspace(N, d, V, T, chunk, kind="projected_backward")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fckl.projected_logprobs_backward(*args, chunk=chunk, round_dW=True, ws=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert fckl.check(ws) == fckl.OK and all(torch.equal(a, b) for a, b in zip(got, want))
    g.mul_(-0.5)
    want = fckl.projected_logprobs_backward(*args, chunk=chunk, round_dW=True)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_projected_dW_rounding_rule(fckl, monkeypatch):
    """A shape at which the library takes the second stream by itself (2 rows d V of 6e11)."""
    N, d, V = 600, 2048, 250000
    Ht, Wt, tokens = make(N, d, V, 1, "bf16", 22)
    _, ent, lse = fckl.projected_logprobs(Ht, Wt, tokens, 600)
    g = torch.randn(N, 1, device="cuda")
    args = (Ht, Wt, tokens, lse, ent, g)
    monkeypatch.delenv("FCKL_OVERLAP", raising=False)
    a = fckl.projected_logprobs_backward(*args, chunk=600, round_dW=True)
    monkeypatch.setenv("FCKL_OVERLAP", "0")
    b = fckl.projected_logprobs_backward(*args, chunk=600, round_dW=True)
    assert fckl.check() == fckl.OK and all(torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------------------------ limits of the decoding form
def launches(fckl, call):
    """Launches of the call by kernel."""
    fckl.profile_enable(True)
    fckl.profile_read()
    out = call()
    torch.cuda.synchronize()
    counts = {k: n for k, (_, n) in fckl.profile_read().items() if n}
    fckl.profile_enable(False)
    return out, counts


@gpu
@pytest.mark.parametrize("N,d,V,T,decoding", [
    (15, 64, 333, 1, True), (16, 256, 4097, 1, True), (17, 256, 4097, 1, False),  # positions
    (16, 64, 33, 32, True), (16, 64, 333, 33, False), (10, 1000, 16, 32, True),   # tokens
    (16, 1408, 700, 32, True), (16, 1416, 700, 32, False),                        # shared memory
    (16, 1472, 501, 1, True), (16, 1480, 501, 1, False),
    (8, 3520, 501, 1, True), (8, 3528, 501, 1, False), (9, 72, 15, 4, True),
])
def test_projected_decode_limits(fckl, N, d, V, T, decoding):
    """Both sides of each limit of the decoding form, and which form ran."""
    Ht, Wt, tokens = make(N, d, V, T, "bf16", seed=N + V + T)
    (logp, ent, lse), ran = launches(fckl, lambda: fckl.projected_logprobs(Ht, Wt, tokens, 2048))
    assert fckl.check() == fckl.OK
    assert ("head_skinny" in ran) == decoding and ("head_logits_stats" in ran) != decoding, ran
    H, W = exact_inputs(Ht, Wt)
    w_logp, w_ent, w_lse = orc.projected(H, W, tokens.cpu().numpy())
    dz, r = logit_error(H, W), (256 + V // 16 + 80) * U + 2.0 ** -21
    close(f64(lse), w_lse, dz + r + 8 * U * np.abs(w_lse))
    close(f64(logp), w_logp, (2 * dz + r)[:, None] + 8 * U * np.abs(w_logp))
    spread = np.maximum(w_ent, np.log(V)) + 2
    close(f64(ent), w_ent, (dz * 2 * spread + r * (1 + 2 * spread)))


# ------------------------------------------------------------------ one token for many positions
@gpu
@pytest.mark.parametrize("N,d,T,chunk,ids", [
    (2, 1544, 1, 2, 1), (3, 1544, 2, 2, 1), (40, 1544, 1, 40, 2), (90, 2056, 3, 64, 5), (700, 1032, 1, 512, 1),
    (600, 520, 8, 600, 3), (5, 512, 1, 5, 1), (5, 520, 1, 5, 1),
])
def test_projected_entries_of_one_token(fckl, N, d, T, chunk, ids):
    """Positions that score the same few tokens (a yes/no judgement, an end of text): the columns of a
    token's row of dW are shared among blocks, fewer and more of them than the token has entries, and
    entries of several windows meet in a row. dW as fp32, dH to bf16, both as exact as elsewhere."""
    V = 600
    Ht, Wt, tokens = make(N, d, V, T, "bf16", seed=N + d)
    tokens = torch.where(tokens < 0, tokens, tokens % ids * 7)
    _, ent, lse = fckl.projected_logprobs(Ht, Wt, tokens, chunk)
    g = torch.randn(N, T, device="cuda")
    dH, dW = fckl.projected_logprobs_backward(Ht, Wt, tokens, lse, ent, g, chunk=chunk)
    assert fckl.check() == fckl.OK
    H, W = exact_inputs(Ht, Wt)
    tk, gn = tokens.cpu().numpy(), f64(g)
    gn = np.where(tk < 0, 0, gn)
    G = orc.logits_gradient(H @ W.T, tk, gn)
    q = np.exp(orc._log_softmax(H @ W.T)[0])
    a = np.abs(gn).sum(1, keepdims=True)
    dz, r = logit_error(H, W)[:, None], (256 + 92) * U + 2.0 ** -21
    eG = q * a * (2.0 ** -8 * 1.01 + 4 * (dz + r) + 2.0 ** -19) + 8 * U * a * (G != 0)
    sums = 4 * max(N * T, V // 16) * U
    close(f64(dW), G.T @ H, eG.T @ np.abs(H) + sums * (np.abs(G).T @ np.abs(H)) + 1e-30)
    want = G @ W
    close(f64(dH), want, eG @ np.abs(W) + sums * (np.abs(G) @ np.abs(W)) + 2.0 ** -8 * np.abs(want) + 1e-30)
    again = fckl.projected_logprobs_backward(Ht, Wt, tokens, lse, ent, g, chunk=chunk)
    assert torch.equal(again[0], dH) and torch.equal(again[1], dW)
