"""Scoring of logits at hand (token_logprobs and its gradient) against the fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32):
* The statistics are fp32 sums: a thread adds at most n = ceil(V / (256 * split)) + 32 values one
  after the other and the merges add ten more, each term within 2^-21 of its own value (2^y to
  2^-22, y = (z - m) log2 e rounded twice, |y| e^{-|y|} < 1): a relative error of at most
  (n + 42) u + 2^-21 =: r of the sums. log s is off by r, a log-probability by r + 4 u |logp|, the
  entropy by r (1 + 2 E) with E = max(entropy, log V).
* A gradient entry is off by |q| (|a| + |ge log q| + |ge|) (4 r + 2^-20) and half a step of its
  type (bf16 2^-8 relative counted on the value, fp16 2^-11 and half its smallest subnormal).
Ids have to be equal.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import scoring_oracle as orc

gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24


def make(N, V, T, dtype, seed, mask="none", scale=3.0, pad=0, offset=0):
    """(logits on the GPU as a view with `pad` columns of NaN between rows and `offset` elements
    before the first, tokens, the logits as fp64)."""
    rng = np.random.default_rng(seed)
    z = rng.normal(size=(N, V)) * scale
    tokens = rng.integers(0, V, size=(N, T))
    tokens[rng.random((N, T)) < 0.1] = -1
    if mask != "none":
        keep = rng.random((N, V)) < 0.02
        if N > 1:
            keep[N // 2] = False  # nothing left
        low = -np.inf if mask == "inf" else torch.finfo(DT[dtype]).min
        z[~keep] = low
    return place(torch.from_numpy(z).to(DT[dtype]), pad, offset), torch.from_numpy(tokens).int().cuda()


def place(z, pad=0, offset=0):
    N, V = z.shape
    buf = torch.full((offset + N * (V + pad) + 8,), float("nan"), dtype=z.dtype, device="cuda")
    view = buf[offset:offset + N * (V + pad)].view(N, V + pad)[:, :V]
    view.copy_(z)
    return view


def f64(t):
    return t.detach().cpu().double().numpy()


def rel_sum(V):
    return (-(-V // 256) + 74) * U + 2.0 ** -21


def close(got, want, tol):
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        bad = ~(same | (np.abs(got - want) <= tol))
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], np.broadcast_to(tol, got.shape)[bad][:4])


def check_scores(fckl, z, tokens, top, got=None):
    logp, ent, norm, ids, lps = got or fckl.token_logprobs(z, tokens, top=top)
    assert fckl.check() == fckl.OK
    zz, r = f64(z), rel_sum(z.shape[1])
    w_logp, w_ent, w_m, w_s = orc.score(zz, tokens.cpu().numpy())
    close(f64(logp), w_logp, r + 4 * U * np.abs(np.where(np.isfinite(w_logp), w_logp, 0)))
    E = np.maximum(w_ent, np.log(z.shape[1]))
    close(f64(ent), w_ent, r * (1 + 2 * E))
    close(f64(norm)[:, 0], w_m, 0)
    close(f64(norm)[:, 1], w_s, r + 4 * U * np.abs(w_s))
    assert tuple(ids.shape) == tuple(lps.shape) == (z.shape[0], top)
    if top:
        w_ids, w_lps = orc.alternatives(zz, top)
        assert np.array_equal(ids.cpu().numpy(), w_ids)
        close(f64(lps), w_lps, r + 4 * U * np.abs(np.where(np.isfinite(w_lps), w_lps, 0)))


@gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("N,V,T,top", [
    (1, 1, 1, 1), (3, 2, 2, 2), (5, 7, 1, 7), (2, 8, 0, 3), (4, 33, 5, 0), (1, 1000, 3, 1000),
    (9, 1024, 1, 1024), (7, 4099, 2, 20), (160, 2500, 1, 5), (3, 32771, 4, 100), (1, 128256, 1, 20), (2, 65537, 1, 1024),
    (20, 40000, 8, 64), (330, 9001, 2, 100),
])
def test_scores(fckl, dtype, N, V, T, top):
    z, tokens = make(N, V, T, dtype, seed=N + V)
    check_scores(fckl, z, tokens, top)


@gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 5), (8, 8), (13, 2)])
def test_scores_strides_and_alignment(fckl, dtype, pad, offset):
    """Rows off the 16-byte boundary, and NaN before, between and after them, never read."""
    z, tokens = make(6, 3001, 2, dtype, seed=pad, pad=pad, offset=offset)
    assert z.stride(0) == 3001 + pad
    check_scores(fckl, z, tokens, 33)


@gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("mask", ["inf", "lowest"])
@pytest.mark.parametrize("N,V,top", [(5, 5003, 30), (1, 40001, 200), (200, 3000, 128)])
def test_scores_masked(fckl, dtype, mask, N, V, top):
    """Masked tokens among the alternatives, rows with nothing left, fewer tokens left than top."""
    z, tokens = make(N, V, 3, dtype, seed=7, mask=mask)
    check_scores(fckl, z, tokens, top)


@gpu
@pytest.mark.parametrize("N", [1, 3, 400])
@pytest.mark.parametrize("V,top", [(50000, 100), (50000, 1024), (3000, 1024)])
def test_alternatives_ties(fckl, N, V, top):
    """Equal logits come by id: a coarse grid of values, a constant row, zeros of both signs, few
    distinct values, long runs in order (more candidates than fit), one peak."""
    rng = np.random.default_rng(V + top)
    rows = [np.round(rng.normal(size=V) * 2) / 2, np.full(V, -3.25), np.where(rng.random(V) < 0.5, 0.0, -0.0),
            (rng.random(V) < 0.001) * 4.0, np.sort(rng.normal(size=V)), -np.sort(rng.normal(size=V)),
            np.minimum(np.arange(V) // 3, 9000) / 64.0, np.eye(1, V, V // 2)[0] * 30,
            np.where(np.arange(V) < 2 * top, 5.0, rng.normal(size=V)),
            np.where(np.arange(V) >= V - top - 7, 5.0, -np.inf)]
    z = np.stack([rows[i % len(rows)] for i in range(N)]) if N > 1 else np.stack(rows[:1])
    if N == 3:
        z = np.stack(rows)  # all kinds
    zt = place(torch.from_numpy(z).float())
    check_scores(fckl, zt, torch.zeros(len(z), 1, dtype=torch.int32, device="cuda"), top)


@gpu
@pytest.mark.parametrize("N", [1, 300])
def test_long_rows(fckl, N):
    """Rows with more vectors than group maxima fit in a block: a group spans several steps."""
    V = 600001
    z = (torch.randn(N, V, device="cuda", generator=torch.Generator("cuda").manual_seed(3)) * 3).bfloat16()
    tokens = torch.randint(0, V, (N, 2), device="cuda", dtype=torch.int32)
    got = fckl.token_logprobs(z, tokens, top=50)
    pick = [0, N // 2, N - 1]
    check_scores(fckl, z[pick], tokens[pick], 50, got=tuple(t[pick] for t in got))


@gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("N,V,top,mask", [
    (500, 1, 1, "none"), (460, 9, 3, "inf"), (500, 300, 64, "lowest"), (500, 301, 65, "none"), (470, 2041, 64, "none"),
    (460, 4100, 64, "inf"), (457, 2001, 100, "inf"), (500, 8190, 128, "none"), (456, 5003, 40, "lowest"),
    (160, 8200, 64, "none"), (160, 3000, 0, "inf"), (458, 33000, 2, "none"),
])
def test_scores_many_rows(fckl, dtype, N, V, top, mask):
    """More rows than SMs hold: blocks of 64 and 128 threads, on both sides of their limits."""
    z, tokens = make(N, V, 2, dtype, seed=N + V + top, mask=mask, pad=V % 3, offset=V % 2)
    check_scores(fckl, z, tokens, top)


@gpu
@pytest.mark.parametrize("N,V,top,mask", [(1216, 48005, 100, "none"), (1300, 48001, 0, "inf"), (160, 100003, 20, "lowest"),
                                          (456, 100001, 600, "none"), (1217, 60000, 1024, "inf")])
def test_scores_many_long_fp32_rows(fckl, N, V, top, mask):
    """Rows that pass through shared memory; a few of them against the oracle."""
    rng = torch.Generator("cuda").manual_seed(N)
    z = torch.randn(N, V + 3, device="cuda", generator=rng)[:, 2:2 + V]
    if mask != "none":
        low = -float("inf") if mask == "inf" else torch.finfo(torch.float32).min
        z.masked_fill_(torch.rand(N, V, device="cuda", generator=rng) > 0.02, low)
        z[N - 1] = low
    tokens = torch.randint(0, V, (N, 2), device="cuda", dtype=torch.int32, generator=rng)
    got = fckl.token_logprobs(z, tokens, top=top)
    pick = [0, 1, 2, 3, N // 2, N - 2, N - 1]
    check_scores(fckl, z[pick], tokens[pick], top, got=tuple(t[pick] for t in got))


@gpu
@pytest.mark.parametrize("V,top", [(1500, 60), (1500, 128), (6000, 64), (6000, 128)])
def test_alternatives_ties_many_rows(fckl, V, top):
    rng = np.random.default_rng(V + top)
    rows = [np.round(rng.normal(size=V) * 2) / 2, np.full(V, -3.25), np.where(rng.random(V) < 0.5, 0.0, -0.0),
            (rng.random(V) < 0.001) * 4.0, np.sort(rng.normal(size=V)), -np.sort(rng.normal(size=V)),
            np.minimum(np.arange(V) // 3, 9000) / 64.0, np.where(np.arange(V) < 2 * top, 5.0, rng.normal(size=V)),
            np.where(np.arange(V) >= V - top - 7, 5.0, -np.inf), np.full(V, -np.inf)]
    z = np.stack([rows[i % len(rows)] for i in range(500)])
    z[11, 3], z[24, V - 1] = np.nan, np.inf
    tokens = torch.zeros(500, 1, dtype=torch.int32, device="cuda")
    got = fckl.token_logprobs(torch.from_numpy(z).float().cuda(), tokens, top=top)
    assert torch.isnan(got[0][[11, 24]]).all() and torch.isnan(got[4][[11, 24]]).all()
    keep = [i for i in range(500) if i not in (11, 24)]
    check_scores(fckl, torch.from_numpy(z[keep]).float().cuda(), tokens[keep], top, got=tuple(t[keep] for t in got))


@gpu
def test_scores_of_extreme_rows(fckl):
    """NaN and +inf make their own row NaN (alternatives 0..top-1) and no other; large offsets and
    a lone finite value are exact."""
    V = 3000
    z = torch.randn(8, V, device="cuda")
    z[1, 17] = float("nan")
    z[2, 2999] = float("inf")
    z[3] = -float("inf")
    z[4] = -float("inf")
    z[4, 1234] = -7.0
    z[5] += 30000.0
    z[6] = -float("inf")
    z[6, 5] = float("nan")
    tokens = torch.full((8, 1), 1234, dtype=torch.int32, device="cuda")
    logp, ent, norm, ids, lps = fckl.token_logprobs(z, tokens, top=4)
    assert fckl.check() == fckl.OK
    for n in (1, 2, 6):
        assert torch.isnan(logp[n]).all() and torch.isnan(ent[n]) and torch.isnan(lps[n]).all()
        assert ids[n].tolist() == [0, 1, 2, 3]
    keep = [0, 3, 4, 5, 7]
    check_scores(fckl, z[keep], tokens[keep], 4, got=tuple(t[keep] for t in (logp, ent, norm, ids, lps)))
    assert logp[4, 0] == 0 and ent[4] == 0 and ids[4, 0] == 1234


@gpu
def test_empty_calls(fckl):
    z = torch.empty(0, 50, device="cuda")
    out = fckl.token_logprobs(z, torch.empty(0, 2, dtype=torch.int32, device="cuda"), top=3)
    assert [tuple(t.shape) for t in out] == [(0, 2), (0,), (0, 2), (0, 3), (0, 3)]
    d = fckl.token_logprobs_backward(z, torch.empty(0, 2, dtype=torch.int32, device="cuda"), out[2], out[1], out[0])
    assert tuple(d.shape) == (0, 50)


@gpu
def test_bad_token_reported(fckl):
    z = torch.randn(3, 100, device="cuda")
    tokens = torch.tensor([[5], [100], [-2]], dtype=torch.int32, device="cuda")
    ws = fckl.Workspace.status()
    logp = fckl.token_logprobs(z, tokens, ws=ws)[0]
    assert fckl.check(ws, raise_on_error=False) == fckl.ERR_INDEX
    assert torch.isfinite(logp[0]).all() and torch.isnan(logp[1:]).all()
    assert fckl.check(ws) == fckl.OK  # read and cleared
    ok = torch.tensor([[5], [99], [-1]], dtype=torch.int32, device="cuda")
    fckl.token_logprobs(z, ok, ws=ws)
    assert fckl.check(ws) == fckl.OK


# ------------------------------------------------------------------ gradient
def grad_tolerance(zz, tokens, g, ge, want, dtype):
    lq = orc._log_softmax(zz)[0]
    q = np.exp(lq)
    lq = np.where(q > 0, lq, 0)
    gg = np.where(tokens < 0, 0, g)
    ent = -(q * lq).sum(1, keepdims=True)
    a = np.abs(gg).sum(1, keepdims=True) + np.abs(ge[:, None]) * (1 + np.abs(lq) + ent)
    half = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -23}[dtype]
    tiny = {"bf16": 1e-38, "fp16": 2.0 ** -25, "fp32": 1e-38}[dtype]
    return q * a * (4 * rel_sum(zz.shape[1]) * (1 + ent) + 2.0 ** -20) + half * np.abs(want) + tiny + \
        8 * U * np.abs(gg).sum(1, keepdims=True) * (np.abs(want) > q * a)


@gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("N,V,T,mask,pad,offset,with_entropy", [
    (1, 1, 1, "none", 0, 0, True), (3, 9, 4, "none", 0, 0, True), (4, 4099, 1, "none", 1, 3, True),
    (3, 40000, 40, "none", 0, 0, False), (5, 5003, 3, "inf", 0, 1, True), (5, 5003, 3, "lowest", 2, 0, True),
    (2, 300, 1024, "none", 0, 0, True), (4, 2500, 0, "none", 0, 0, True), (65, 16391, 2, "none", 0, 0, True),
])
def test_gradient(fckl, dtype, N, V, T, mask, pad, offset, with_entropy):
    z, tokens = make(N, V, T, dtype, seed=V, mask=mask, pad=pad, offset=offset)
    rng = np.random.default_rng(V + 1)
    g = rng.normal(size=(N, T)).astype(np.float32)
    ge = rng.normal(size=N).astype(np.float32) if with_entropy else np.zeros(N, np.float32)
    _, ent, norm, _, _ = fckl.token_logprobs(z, tokens)
    gt = torch.from_numpy(g).cuda()
    got = fckl.token_logprobs_backward(z, tokens, norm, ent, gt, torch.from_numpy(ge).cuda() if with_entropy else None)
    assert fckl.check() == fckl.OK and got.dtype == z.dtype
    zz, tk = f64(z), tokens.cpu().numpy()
    want = orc.logits_gradient(zz, tk, g, ge)
    close(f64(got), want, grad_tolerance(zz, tk, g, ge, want, dtype))
    # in place, and into rows of another alignment: the same bits
    zc = place(z, pad, offset)
    inplace = fckl.token_logprobs_backward(zc, tokens, norm, ent, gt,
                                           torch.from_numpy(ge).cuda() if with_entropy else None, out=zc)
    assert inplace.data_ptr() == zc.data_ptr() and torch.equal(inplace, got)
    other = place(torch.zeros_like(z), pad + 1, offset + 1)
    fckl.token_logprobs_backward(z, tokens, norm, ent, gt, torch.from_numpy(ge).cuda() if with_entropy else None,
                                 out=other)
    assert torch.equal(other, got)


@gpu
@pytest.mark.parametrize("N,V,T", [(4, 32761, 3), (4, 32765, 2), (3, 65530, 2), (2, 900, 512), (2, 900, 513), (700, 8197, 1)])
def test_gradient_block_sizes(fckl, N, V, T):
    """Both sides of the row length and the number of tokens up to which blocks are smaller."""
    for dtype in ("bf16", "fp32"):
        z, tokens = make(N, V, T, dtype, seed=V, pad=1, offset=1)
        rng = np.random.default_rng(V + T)
        g, ge = rng.normal(size=(N, T)).astype(np.float32), rng.normal(size=N).astype(np.float32)
        _, ent, norm, _, _ = fckl.token_logprobs(z, tokens)
        got = fckl.token_logprobs_backward(z, tokens, norm, ent, torch.from_numpy(g).cuda(), torch.from_numpy(ge).cuda())
        zz, tk = f64(z), tokens.cpu().numpy()
        want = orc.logits_gradient(zz, tk, g, ge)
        close(f64(got), want, grad_tolerance(zz, tk, g, ge, want, dtype))


@gpu
@pytest.mark.parametrize("mask", ["inf", "lowest"])
def test_gradient_of_masked_logits_under_large_upstreams(fckl, mask):
    """Upstream gradients of 2^60 (a loss scale, say): masked places stay 0, the rest finite."""
    z, tokens = make(5, 5003, 3, "fp32", seed=4, mask=mask)
    scale = 2.0 ** 60
    rng = np.random.default_rng(5)
    g, ge = (rng.normal(size=s).astype(np.float32) * np.float32(scale) for s in ((5, 3), (5,)))
    _, ent, norm, _, _ = fckl.token_logprobs(z, tokens)
    got = f64(fckl.token_logprobs_backward(z, tokens, norm, ent, torch.from_numpy(g).cuda(), torch.from_numpy(ge).cuda()))
    zz, tk = f64(z), tokens.cpu().numpy()
    want = orc.logits_gradient(zz, tk, g, ge)
    close(got / scale, want / scale, grad_tolerance(zz, tk, g / scale, ge / scale, want / scale, "fp32"))


@gpu
def test_gradient_of_rows_without_upstream_is_zero(fckl):
    """Positions that the loss leaves out may hold NaN; nothing of it reaches the gradient."""
    z = torch.randn(4, 1000, device="cuda")
    z[1] = float("nan")
    z[2, 3] = float("inf")
    tokens = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    tokens[3] = -1
    _, ent, norm, _, _ = fckl.token_logprobs(z, tokens)
    g = torch.ones(4, 2, device="cuda")
    g[1:3] = 0
    d = fckl.token_logprobs_backward(z, tokens, norm, ent, g, torch.zeros(4, device="cuda"))
    assert torch.isfinite(d).all() and (d[1:] == 0).all() and (d[0] != 0).any()


@gpu
def test_autograd_matches_differences(fckl):
    """Broadcast and missing upstream gradients through autograd; central differences of the oracle's
    fp64 value along random directions, at fp32 logits."""
    z, tokens = make(6, 700, 3, "fp32", seed=5)
    z = z.clone().requires_grad_()
    logp, ent = fckl.differentiable_token_logprobs(z, tokens)
    (logp.sum() + 0.5 * ent.sum()).backward()
    grad = f64(z.grad)
    rng = np.random.default_rng(0)
    zz, tk = f64(z), tokens.cpu().numpy()

    def value(x):
        a, b, _, _ = orc.score(x, tk)
        return a.sum() + 0.5 * b.sum()

    for _ in range(5):
        v = rng.normal(size=zz.shape)
        diff = (value(zz + 1e-5 * v) - value(zz - 1e-5 * v)) / 2e-5
        # fp32 gradient entries, each within 2^-18 of the row's upstream sum; differences to 1e-8
        assert abs(diff - (grad * v).sum()) <= 2.0 ** -18 * np.abs(v).sum() / 100 + 1e-6 * abs(diff) + 1e-6
    z.grad = None
    fckl.differentiable_token_logprobs(z, tokens)[1].sum().backward()  # entropy alone
    want = orc.logits_gradient(zz, tk, np.zeros(tk.shape), np.ones(6))
    close(f64(z.grad), want, grad_tolerance(zz, tk, np.zeros(tk.shape), np.ones(6), want, "fp32"))


@gpu
def test_other_stream_and_graph(fckl):
    z, tokens = make(40, 5000, 2, "bf16", seed=11)
    want = fckl.token_logprobs(z, tokens, top=10)
    g = torch.randn(40, 2, device="cuda")
    dwant = fckl.token_logprobs_backward(z, tokens, want[2], want[1], g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = fckl.token_logprobs(z, tokens, top=10, stream=side)
    dgot = fckl.token_logprobs_backward(z, tokens, got[2], got[1], g, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(dgot, dwant)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gout = fckl.token_logprobs(z, tokens, top=10)
        gd = fckl.token_logprobs_backward(z, tokens, gout[2], gout[1], g)
    z2, t2 = make(40, 5000, 2, "bf16", seed=12)
    z.copy_(z2)
    tokens.copy_(t2)
    graph.replay()
    torch.cuda.synchronize()
    want = fckl.token_logprobs(z2, t2, top=10)
    assert all(torch.equal(a, b) for a, b in zip(gout, want))
    assert torch.equal(gd, fckl.token_logprobs_backward(z2, t2, want[2], want[1], g))


@gpu
def test_offsets_past_32_bits(fckl):
    """More than 2^31 logits: the last rows match the same rows scored on their own, bit for bit."""
    N, V = 70000, 32000
    z = torch.empty(N, V, dtype=torch.bfloat16, device="cuda")
    z.normal_(generator=torch.Generator("cuda").manual_seed(1)).mul_(3)
    tokens = torch.randint(0, V, (N, 1), device="cuda", dtype=torch.int32)
    got = fckl.token_logprobs(z, tokens, top=5)
    g = torch.ones(N, 1, device="cuda")
    tail = slice(N - 400, N)  # both sides with one block per row
    own = fckl.token_logprobs(z[tail].clone(), tokens[tail].contiguous(), top=5)
    assert all(torch.equal(a[tail], b) for a, b in zip(got, own))
    d = fckl.token_logprobs_backward(z, tokens, got[2], got[1], g)
    down = fckl.token_logprobs_backward(z[tail].clone(), tokens[tail].contiguous(), own[2], own[1], g[tail])
    assert torch.equal(d[tail], down)
    check_scores(fckl, z[tail][:3], tokens[tail][:3].contiguous(), 5, got=tuple(t[tail][:3] for t in got))


# ------------------------------------------------------------------ refusals (CPU)
def test_argument_errors_launch_nothing(fckl):
    lib = fckl.load()
    before = lib.fckl_launch_count()
    p, z = ctypes.c_void_p(256), ctypes.c_void_p(0)

    def fwd(logits=p, dt=0, ld=100, tokens=p, N=4, V=100, T=2, top=3, logp=p, ent=p, norm=p, ti=p, tl=p, ws=p, n=256):
        return lib.fckl_token_logprobs(logits, dt, ld, tokens, N, V, T, top, logp, ent, norm, ti, tl, ws, n, z)

    odd = ctypes.c_void_p(257)
    for bad in (dict(N=-1), dict(V=0), dict(T=-1), dict(top=-1), dict(ld=99), dict(dt=3), dict(dt=-1),
                dict(logits=z), dict(logits=odd), dict(logits=ctypes.c_void_p(258), dt=1), dict(tokens=z),
                dict(tokens=odd), dict(logp=z), dict(ent=z), dict(norm=odd), dict(ti=z), dict(tl=z), dict(ws=z),
                dict(ws=ctypes.c_void_p(128))):
        assert fwd(**bad) == fckl.ERR_ARG, bad
    for bad in (dict(T=1025), dict(top=101), dict(V=2000, ld=2000, top=1025), dict(V=(1 << 30) + 1, ld=1 << 31),
                dict(N=(1 << 40) + 1)):
        assert fwd(**bad) == fckl.ERR_UNSUPPORTED, bad
    assert fwd(n=255) == fckl.ERR_WORKSPACE
    assert fwd(N=0, logits=z, tokens=z, logp=z, ent=z, norm=z, ti=z, tl=z) == fckl.OK

    def bwd(logits=p, dt=0, ld=100, tokens=p, N=4, V=100, T=2, norm=p, ent=p, g=p, ge=z, out=ctypes.c_void_p(4096),
            ldo=100, ws=p, n=256):
        return lib.fckl_token_logprobs_backward(logits, dt, ld, tokens, N, V, T, norm, ent, g, ge, out, ldo, ws, n, z)

    for bad in (dict(ldo=99), dict(norm=z), dict(ent=z), dict(g=z), dict(out=z), dict(out=odd), dict(ge=odd),
                dict(out=p, ldo=101), dict(dt=7)):
        assert bwd(**bad) == fckl.ERR_ARG, bad
    assert bwd(n=0) == fckl.ERR_WORKSPACE
    assert bwd(N=0) == fckl.OK
    assert lib.fckl_launch_count() == before


@pytest.mark.parametrize("bad", [
    lambda f, z, t: f.token_logprobs(z.double(), t), lambda f, z, t: f.token_logprobs(z, t.long()),
    lambda f, z, t: f.token_logprobs(z[0], t), lambda f, z, t: f.token_logprobs(z, t[:2]),
    lambda f, z, t: f.token_logprobs(z.t().contiguous().t(), t), lambda f, z, t: f.token_logprobs(z[:1].expand(3, 8), t),
    lambda f, z, t: f.token_logprobs(z, t), lambda f, z, t: f.token_logprobs(z, t.t().contiguous().t()),
    lambda f, z, t: f.token_logprobs_backward(z, t, z, z[:, 0], z),
])
def test_binding_refusals(fckl, bad):
    """Wrong types, shapes and layouts, and tensors that are not on the GPU."""
    z, t = torch.zeros(3, 8), torch.zeros(3, 2, dtype=torch.int32)
    with pytest.raises((TypeError, ValueError)):
        bad(fckl, z, t)


# ------------------------------------------------------------------ the largest numbers of a type
def far_rows(V, dtype):
    """Rows with finite logits up to the type's largest: a forced token (set to the largest number, as the
    mirror image of a mask) beside ordinary, -inf and lowest ones, several, all, and just below."""
    info = torch.finfo(DT[dtype])
    rng = np.random.default_rng(V)
    z = rng.normal(size=(9, V)) * 3
    z[0, V // 2] = info.max
    z[1, [0, V // 3, V - 1]] = info.max
    z[2] = -np.inf
    z[2, V // 2] = info.max
    z[3] = info.min
    z[3, V // 2] = info.max
    z[4, V // 2] = 0.7 * info.max
    z[5] = info.max
    z[6, ::3], z[6, 1::3] = -np.inf, info.min
    z[6, V // 2] = info.max
    z[7, V // 2], z[7, 0] = 0.5 * info.max, -0.5 * info.max
    z[8] *= info.max / 64
    return z


@gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("N,V,top", [(9, 1, 1), (9, 3001, 5), (9, 40003, 300), (504, 1500, 20), (504, 20011, 2),
                                     (1224, 48005, 3)])
def test_finite_logits_of_any_size(fckl, dtype, N, V, top):
    """Finite logits give finite statistics, and gradients, however large they are; with blocks of every
    size, rows over several blocks, and rows through shared memory. A log-probability past the largest
    fp32 number is -inf."""
    nine = torch.from_numpy(far_rows(V, dtype)).to(DT[dtype])
    zz = nine.double().numpy()
    z = nine.cuda().repeat(N // 9, 1)
    rng = np.random.default_rng(1)
    tk = np.stack([np.full(9, V // 2), rng.integers(0, V, 9)], 1)
    tokens = torch.from_numpy(tk).int().cuda().repeat(N // 9, 1)
    got = fckl.token_logprobs(z, tokens, top=top)
    assert fckl.check() == fckl.OK
    for t in got:  # whichever rows of the batch: the same bits
        assert all(torch.equal(t[:9], t[i:i + 9]) for i in range(9, N, 9))
    logp, ent, norm, ids, lps = (t[:9] for t in got)
    with np.errstate(over="ignore"):
        w_logp, w_ent, w_m, w_s = (a.astype(np.float32).astype(np.float64) for a in orc.score(zz, tk))
        w_ids, w_lps = orc.alternatives(zz, top)
        w_lps = w_lps.astype(np.float32).astype(np.float64)
    r = rel_sum(V)
    close(f64(logp), w_logp, r + 5 * U * np.abs(np.where(np.isfinite(w_logp), w_logp, 0)))
    close(f64(ent), w_ent, r * (1 + 2 * np.maximum(w_ent, np.log(V))))
    close(f64(norm)[:, 0], w_m, 0)
    close(f64(norm)[:, 1], w_s, r + 4 * U * np.abs(w_s))
    assert np.array_equal(ids.cpu().numpy(), w_ids)
    close(f64(lps), w_lps, r + 5 * U * np.abs(np.where(np.isfinite(w_lps), w_lps, 0)))
    g = rng.normal(size=(9, 2)).astype(np.float32)
    for ge in (rng.normal(size=9).astype(np.float32), np.zeros(9, np.float32), None):
        gt = torch.from_numpy(g).cuda().repeat(N // 9, 1)
        get = None if ge is None else torch.from_numpy(ge).cuda().repeat(N // 9)
        d = fckl.token_logprobs_backward(z, tokens, got[2], got[1], gt, get)
        assert torch.equal(d[:9], d[-9:])
        g0 = np.zeros(9) if ge is None else ge
        want = orc.logits_gradient(zz, tk, g, g0)
        close(f64(d[:9]), want, grad_tolerance(zz, tk, g, g0, want, dtype))


@gpu
@pytest.mark.parametrize("dtype", list(DT))
def test_gradient_without_entropy_does_not_read_it(fckl, dtype):
    """Where no gradient comes in through the entropy, what stands in its place does not matter."""
    z, tokens = make(6, 3001, 2, dtype, seed=2)
    _, ent, norm, _, _ = fckl.token_logprobs(z, tokens)
    g = torch.randn(6, 2, device="cuda")
    want = fckl.token_logprobs_backward(z, tokens, norm, ent, g)
    nothing = torch.full_like(ent, float("nan"))
    assert torch.isfinite(want).all()
    assert torch.equal(fckl.token_logprobs_backward(z, tokens, norm, nothing, g), want)
    assert torch.equal(fckl.token_logprobs_backward(z, tokens, norm, nothing, g, torch.zeros(6, device="cuda")), want)
    ge = torch.zeros(6, device="cuda")
    ge[4] = 0.5
    mixed = torch.where(ge == 0, nothing, ent)
    keep = [0, 1, 2, 3, 5]
    assert torch.equal(fckl.token_logprobs_backward(z, tokens, norm, mixed, g, ge),
                       fckl.token_logprobs_backward(z, tokens, norm, ent, g, ge))
    assert torch.equal(fckl.token_logprobs_backward(z, tokens, norm, mixed, g, ge)[keep], want[keep])


@gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("N", [4, 400])
def test_gradient_of_a_nan_row_is_nan(fckl, dtype, N):
    """A position with an upstream gradient whose logits hold a NaN gets a NaN gradient, whatever else
    they hold (nothing but NaN, NaN among -inf); only a position that is -inf throughout gets zeros."""
    z = torch.randn(N, 1200, device="cuda").to(DT[dtype])
    z[0] = float("nan")
    z[1] = -float("inf")
    z[1, 7] = float("nan")
    z[2] = -float("inf")
    tokens = torch.full((N, 1), 3, dtype=torch.int32, device="cuda")
    logp, ent, norm, _, _ = fckl.token_logprobs(z, tokens)
    d = fckl.token_logprobs_backward(z, tokens, norm, ent, torch.ones(N, 1, device="cuda"))
    assert torch.isnan(d[0]).all() and torch.isnan(d[1, 7]) and torch.isnan(d[1]).all()
    assert (d[2] == 0).all() and torch.isfinite(d[3:]).all()


def _logits_call(f, ws, s):
    z = torch.randn(8, 5000, device="cuda")
    f.token_logprobs(z, torch.zeros(8, 1, dtype=torch.int32, device="cuda"), top=5, ws=ws, stream=s)


def _logits_grad_call(f, ws, s):
    z, t = torch.randn(8, 5000, device="cuda"), torch.zeros(8, 1, dtype=torch.int32, device="cuda")
    one = torch.ones(8, 2, device="cuda")
    f.token_logprobs_backward(z, t, one, one[:, 0].contiguous(), one[:, :1].contiguous(), ws=ws, stream=s)


def _head_call(f, ws, s):
    H, W = torch.ones(8, 64, device="cuda").bfloat16(), torch.ones(900, 64, device="cuda").bfloat16()
    f.projected_logprobs(H, W, torch.zeros(8, 1, dtype=torch.int32, device="cuda"), 8, ws=ws, stream=s)


def _head_grad_call(f, ws, s):
    H, W = torch.ones(8, 64, device="cuda").bfloat16(), torch.ones(900, 64, device="cuda").bfloat16()
    one = torch.ones(8, 1, device="cuda")
    f.projected_logprobs_backward(H, W, torch.zeros(8, 1, dtype=torch.int32, device="cuda"), one[:, 0].contiguous(),
                                  one[:, 0].contiguous(), one, chunk=8, ws=ws, stream=s)


def _matmul_call(f, ws, s):
    a, sa = f.block_quantize(torch.randn(40, 128, device="cuda"))
    b, sb = f.block_quantize(torch.randn(300, 128, device="cuda"), rows=128)
    s.wait_stream(torch.cuda.current_stream())
    f.block_scaled_matmul(a, sa, b, sb, ws=ws, stream=s)


def _projection_call(f, ws, s):
    b, sb = f.block_quantize(torch.randn(300, 128, device="cuda"), rows=128)
    s.wait_stream(torch.cuda.current_stream())
    f.block_scaled_projection(torch.randn(40, 128, device="cuda"), b, sb, ws=ws, stream=s)


@gpu
@pytest.mark.parametrize("call", [_logits_call, _logits_grad_call, _head_call, _head_grad_call, _matmul_call,
                                  _projection_call])
def test_workspace_given_with_a_stream_outlives_its_last_use(fckl, call):
    """A workspace that the caller drops right after a call on another stream is not handed out again
    while that stream still has the call before it."""
    call(fckl, fckl.Workspace.sized(4 << 20, "cuda"), torch.cuda.Stream())  # set-up out of the way
    torch.cuda.synchronize()
    size = 41 << 20
    ws = fckl.Workspace.sized(size, "cuda")
    ws.tensor.zero_()
    torch.cuda.synchronize()
    at = ws.tensor.data_ptr()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # about 0.2 s
    call(fckl, ws, side)
    del ws
    other = torch.empty(size, dtype=torch.uint8, device="cuda")
    busy = not side.query()
    torch.cuda.synchronize()
    assert busy and other.data_ptr() != at
