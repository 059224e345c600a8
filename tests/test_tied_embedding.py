"""The tied embedding (embedding, embedding_backward) against the fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24, h = half a step of the result's type relative to the value,
at least half its smallest subnormal):
* A lookup is one fp32 product, rounded once: u + h of the value (h alone where the type is fp32), and
  the bits of the same two steps on the CPU.
* A gradient is the fp32 sum of a token's n rows: one after the other within at most 64 entries (a warp's
  32, then the four warps of a tile, or a tile of 64), then the tiles' sums (tiles of at least 8 entries):
  at most 64 + n / 8 + 1 additions, never more than n + 1, each off by u of the partial sum, itself at
  most the sum of |g|;
  the scale and the addition to the old value add 2 u of theirs, the result's rounding h.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import training_step_oracle as orc

gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24


def f64(t):
    return t.detach().cpu().double().numpy()


def half_step(want, dtype):
    info = torch.finfo(dtype)
    return np.maximum(np.abs(want) * info.eps / 2, info.smallest_normal * info.eps / 2)


def close(got, want, tol):
    bad = ~((np.abs(got - want) <= tol) | (got == want))
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


def rows(N, d, dtype, seed, pad=0, offset=0, scale=1.0):
    """[N, d] on the GPU as a view with `pad` NaN columns between rows and `offset` before the first."""
    x = torch.from_numpy(np.random.default_rng(seed).normal(size=(N, d)) * scale).to(DT[dtype])
    buf = torch.full((offset + N * (d + pad) + 8,), float("nan"), dtype=x.dtype, device="cuda")
    view = buf[offset:offset + N * (d + pad)].view(N, d + pad)[:, :d]
    view.copy_(x)
    return view


def draw_tokens(N, V, seed, kind="texts"):
    rng = np.random.default_rng(seed)
    if kind == "one":
        t = np.full(N, V - 1)
    elif kind == "empty":
        t = np.full(N, -1)
    elif kind == "different":
        t = rng.permutation(V)[:N] if N <= V else rng.integers(0, V, N)
    else:  # frequent and rare ones, some empty
        t = np.minimum((np.exp(rng.random(N) * np.log(V + 1)) - 1).astype(np.int64), V - 1)
        t = rng.permutation(V)[t]
        t[rng.random(N) < 0.05] = -1
    return torch.from_numpy(t.astype(np.int32)).cuda()


def grad_tolerance(want, size, count, scale, out_dtype, old=None):
    adds = np.minimum(count + 1, 65 + count / 8)[:, None]
    tol = (adds + 2) * U * abs(scale) * size * 1.001 + half_step(want, out_dtype)
    if old is not None:
        tol = tol + 2 * U * (np.abs(old) + np.abs(scale) * size)
    return tol


def check_gradient(fckl, g, tokens, V, scale=1.0, dtype=None, old=None, got=None, ws=None):
    if got is None:
        if old is None:
            got = fckl.embedding_backward(g, tokens, V, scale=scale, dtype=dtype, ws=ws)
        else:
            got = old.clone()
            assert fckl.embedding_backward(g, tokens, V, scale=scale, dW=got, accumulate=True, ws=ws) is got
        assert fckl.check() == fckl.OK
    s = float(np.float32(scale))
    o = None if old is None else f64(old)
    want, size, count = orc.embedding_gradient(f64(g), tokens.cpu().numpy(), V, s, o)
    close(f64(got), want, grad_tolerance(want, size, count, s, got.dtype, o))
    untouched = torch.from_numpy(count == 0).cuda()
    if old is None:
        assert (got[untouched] == 0).all()
    else:
        assert torch.equal(got[untouched], old[untouched])
    return got


# ------------------------------------------------------------------ lookup
@gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("N,d,V", [(1, 1, 1), (1, 2880, 999), (3, 7, 5), (5, 64, 33), (257, 250, 1001), (70, 1028, 400),
                                   (2, 4100, 3), (130, 1022, 77), (1000, 128, 4099)])
def test_lookup(fckl, dtype, N, d, V):
    W, tokens = rows(V, d, dtype, N + d), draw_tokens(N, V, N)
    for scale in (1.0, d ** 0.5, -0.3):
        y = fckl.embedding(W, tokens, scale=scale)
        assert fckl.check() == fckl.OK and y.dtype == W.dtype
        want = orc.embedding(f64(W), tokens.cpu().numpy(), float(np.float32(scale)))
        close(f64(y), want, U * np.abs(want) + half_step(want, y.dtype))
        cpu = W.cpu().float()[tokens.cpu().clamp(min=0).long()] * scale
        cpu[tokens.cpu() < 0] = 0
        assert torch.equal(y.cpu(), cpu.to(y.dtype))


@gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 5), (8, 8), (4, 2)])
@pytest.mark.parametrize("d", [96, 33])
def test_lookup_strides_and_alignment(fckl, dtype, pad, offset, d):
    """Rows apart and off the 16-byte boundary, on both sides; what lies between is neither read nor written."""
    W, tokens = rows(50, d, dtype, 3, pad, offset), draw_tokens(40, 50, 4)
    want = fckl.embedding(W.contiguous(), tokens, scale=2.5)
    assert torch.equal(fckl.embedding(W, tokens, scale=2.5), want)
    buf = torch.full((offset + 40 * (d + pad) + 8,), 7.0, dtype=W.dtype, device="cuda")
    out = buf[offset:offset + 40 * (d + pad)].view(40, d + pad)[:, :d]
    assert fckl.embedding(W, tokens, scale=2.5, out=out) is out
    assert torch.equal(out, want)
    out.fill_(7.0)
    assert (buf == 7.0).all()


@gpu
def test_lookup_shapes_and_bad_ids(fckl):
    W = rows(20, 24, "bf16", 1)
    tokens = torch.tensor([[0, 19, -1], [5, 5, 2]], dtype=torch.int32, device="cuda")
    y = fckl.embedding(W, tokens)
    assert y.shape == (2, 3, 24) and torch.equal(y[1, 0], W[5]) and (y[0, 2] == 0).all()
    assert fckl.embedding(W, tokens[0, 0]).shape == (24,)
    assert fckl.embedding(W, tokens[:, :0].contiguous()).shape == (2, 0, 24)
    assert fckl.check() == fckl.OK
    for bad in (20, -2, 2 ** 31 - 1, -2 ** 31):
        t = torch.tensor([3, bad, 4], dtype=torch.int32, device="cuda")
        y = fckl.embedding(W, t)
        assert fckl.check(raise_on_error=False) == fckl.ERR_INDEX
        assert torch.equal(y[0], W[3]) and torch.isnan(y[1]).all() and torch.equal(y[2], W[4])
        g = torch.ones(3, 24, device="cuda")
        dW = fckl.embedding_backward(g, t, 20)
        assert fckl.check(raise_on_error=False) == fckl.ERR_INDEX
        assert dW.sum() == 48 and (dW[3] == 1).all() and (dW[4] == 1).all()
    assert fckl.check() == fckl.OK


@gpu
def test_lookup_of_extreme_values(fckl):
    """inf, NaN, the largest and the smallest numbers go through one product and one rounding."""
    for dtype in DT.values():
        info = torch.finfo(dtype)
        W = torch.tensor([[float("inf"), -float("inf"), float("nan"), info.max, info.min, info.smallest_normal,
                           info.smallest_normal * info.eps, -0.0]], device="cuda").to(dtype)
        t = torch.zeros(2, dtype=torch.int32, device="cuda")
        for s in (1.0, 2.0, 0.5):
            want = (W.cpu().float() * s).to(dtype)[[0, 0]]
            assert torch.equal(fckl.embedding(W, t, scale=s).cpu().nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))


# ------------------------------------------------------------------ gradient
@gpu
@pytest.mark.parametrize("dtype,out", [("bf16", "fp32"), ("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32")])
@pytest.mark.parametrize("N,d,V,kind", [
    (1, 1, 1, "one"), (1, 2880, 7, "texts"), (7, 8, 3, "texts"), (9, 33, 50, "different"), (64, 40, 64, "one"),
    (65, 40, 3, "empty"), (130, 1030, 513, "texts"), (1000, 24, 2, "texts"), (777, 1022, 100, "texts"),
    (5000, 8, 700, "one"), (9000, 4, 1 << 18, "texts"), (20000, 6, 300, "texts"), (70000, 2, 1000, "texts"),
    (300, 776, 40, "texts"), (260, 2880, 90, "texts"), (129, 1536, 1, "one"), (2000, 96, 7, "texts"),
])
def test_gradient(fckl, dtype, out, N, d, V, kind):
    """Sizes around a warp, a tile and a sorting block, and more positions than one round of the cluster."""
    g, tokens = rows(N, d, dtype, N + d), draw_tokens(N, V, N, kind)
    check_gradient(fckl, g, tokens, V, scale=1.7, dtype=DT[out])
    old = rows(V, d, out, 5).contiguous()
    check_gradient(fckl, g, tokens, V, scale=-0.4, old=old)


@gpu
@pytest.mark.parametrize("V", [1, 2, 511, 512, 513, 1 << 18, (1 << 18) + 1, (1 << 27) + 3])
def test_gradient_vocabulary_sizes(fckl, V):
    """One to four digits of the sort, tokens at both ends."""
    N = 3000
    rng = np.random.default_rng(V)
    t = rng.integers(0, V, N)
    t[:4], t[4:8] = 0, V - 1
    tokens = torch.from_numpy(t.astype(np.int32)).cuda()
    g = torch.from_numpy(rng.integers(-8, 9, size=(N, 2)).astype(np.float32)).cuda()  # sums are exact
    dW = fckl.embedding_backward(g, tokens, V)
    assert fckl.check() == fckl.OK
    want = torch.zeros(V, 2, device="cuda").index_add_(0, tokens.long(), g)
    assert torch.equal(dW, want)


@gpu
@pytest.mark.parametrize("d", [1, 4])
@pytest.mark.parametrize("N", [31, 33, 255, 257, 1023, 1025, 8192, 8193, 65536, 65537, 131073, 300001])
def test_gradient_every_position_once(fckl, N, d):
    """Around the sizes of a warp's entries, of the tiles, of the clusters and of the sort's rounds: exact sums
    of whole numbers, so that a lost or doubled position shows. Frequent and rare tokens, one that takes a
    third of the positions, one alone, and all different; the sums of at most 300001 numbers up to 30 stay
    below 2^24."""
    V = 1237 if N < 1e5 else 1 << 19
    g = torch.arange(N * d, device="cuda", dtype=torch.float32).remainder(61).view(N, d) - 30
    often = draw_tokens(N, V, N)
    often[::3] = V // 2
    for tokens in (draw_tokens(N, V, N), often, draw_tokens(N, V, 1, "one"), draw_tokens(N, V, 1, "different")):
        dW = fckl.embedding_backward(g, tokens, V)
        want = torch.zeros(V, d, device="cuda", dtype=torch.float64)
        want.index_add_(0, tokens.clamp(min=0).long(), torch.where(tokens[:, None] < 0, 0.0, g).double())
        assert torch.equal(dW.double(), want)
        assert torch.equal(fckl.embedding_backward(g, tokens, V), dW)
        old = torch.ones(V, d, device="cuda")
        assert torch.equal(fckl.embedding_backward(g, tokens, V, dW=old, accumulate=True).double(), want + 1)
    assert fckl.check() == fckl.OK


@gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 5), (8, 8)])
@pytest.mark.parametrize("d", [96, 33])
def test_gradient_strides_and_alignment(fckl, dtype, pad, offset, d):
    """Rows apart and off the 16-byte boundary, on both sides. The order of a token's sums depends on the
    alignment, so each layout is held to the tolerance, and the same layout to its bits."""
    g, tokens = rows(200, d, dtype, 3, pad, offset), draw_tokens(200, 50, 4)
    want = check_gradient(fckl, g, tokens, 50)
    check_gradient(fckl, g.contiguous(), tokens, 50)
    assert torch.equal(fckl.embedding_backward(g, tokens, 50), want)
    buf = torch.full((offset + 50 * d + 8,), 7.0, device="cuda")
    dW = buf[offset:offset + 50 * d].view(50, d)
    assert fckl.embedding_backward(g, tokens, 50, dW=dW) is dW
    check_gradient(fckl, g, tokens, 50, got=dW)
    dW.fill_(7.0)
    assert (buf == 7.0).all()


@gpu
def test_gradient_is_deterministic_and_local(fckl):
    """The same call gives the same bits; a NaN or inf stays in its token's row and column; empty slots'
    rows are never read."""
    g, tokens = rows(5000, 72, "bf16", 1).contiguous(), draw_tokens(5000, 400, 2)
    a, b = fckl.embedding_backward(g, tokens, 400), fckl.embedding_backward(g, tokens, 400)
    assert torch.equal(a, b)
    h = g.clone()
    h[tokens == -1] = float("nan")
    assert torch.equal(fckl.embedding_backward(h, tokens, 400), a)
    at = int((tokens >= 0).nonzero()[17])
    h[at, 5], h[at, 6] = float("nan"), float("inf")
    c = fckl.embedding_backward(h, tokens, 400)
    t = int(tokens[at])
    assert torch.isnan(c[t, 5]) and c[t, 6] == float("inf")
    same = torch.ones_like(c, dtype=torch.bool)
    same[t, 5:7] = False
    assert torch.equal(c[same], a[same])


@gpu
def test_gradient_without_positions(fckl):
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    g = torch.empty(0, 16, device="cuda")
    assert (fckl.embedding_backward(g, none, 30, dW=torch.ones(30, 16, device="cuda")) == 0).all()
    old = torch.ones(30, 16, device="cuda")
    assert (fckl.embedding_backward(g, none, 30, dW=old, accumulate=True) == 1).all()
    assert fckl.embedding(old, none).shape == (0, 16)
    assert fckl.check() == fckl.OK


@gpu
def test_offsets_past_32_bits(fckl):
    """More than 2^31 values in W, in dW and in the positions' rows."""
    V, d = 40000, 60000
    W = torch.empty(V, d, dtype=torch.bfloat16, device="cuda")
    W.copy_(torch.arange(V, device="cuda").remainder(251)[:, None])
    tokens = torch.tensor([V - 1, 0, V - 1, 37000], dtype=torch.int32, device="cuda")
    y = fckl.embedding(W, tokens, scale=0.5)
    assert torch.equal(y, (W[tokens.long()].float() * 0.5).bfloat16())
    dW = fckl.embedding_backward(y, tokens, V, dtype=torch.bfloat16)
    assert torch.equal(dW[V - 1], (2 * y[0].float()).bfloat16()) and torch.equal(dW[37000], y[3])
    assert dW.float().sum(1).ne(0).sum() <= 3 and (dW[1:37000] == 0).all() and (dW[37001:V - 1] == 0).all()
    many = torch.arange(V, device="cuda", dtype=torch.int32)  # every row of W as a position
    out = fckl.embedding(W, many)
    assert torch.equal(out, W)
    three = many.remainder(3)
    got = fckl.embedding_backward(out, three, 3)
    want = torch.stack([W[k::3].sum(0, dtype=torch.float32) for k in range(3)])
    assert torch.equal(got, want)  # whole numbers below 2^24: exact in any order


@gpu
@pytest.mark.parametrize("dtype", list(DT))
def test_autograd(fckl, dtype):
    """W's gradient through autograd, of W's type; a broadcast upstream gradient; the gradient against
    differences of the (linear) lookup."""
    W = rows(60, 48, dtype, 1).contiguous().requires_grad_()
    tokens = draw_tokens(96, 60, 3).view(4, 24)
    y = fckl.differentiable_embedding(W, tokens, scale=3.0)
    g = rows(96, 48, dtype, 4).contiguous().view(4, 24, 48)
    dW, = torch.autograd.grad(y, W, g, retain_graph=True)
    assert dW.dtype == W.dtype
    check_gradient(fckl, g, tokens, 60, scale=3.0, got=dW)
    ones, = torch.autograd.grad(y.sum(), W)
    check_gradient(fckl, torch.ones_like(g), tokens, 60, scale=3.0, got=ones)
    # <y(W + D) - y(W), g> = <D, dW> for any D, here in fp32 where both sides are near exact
    if dtype == "fp32":
        D = torch.randn(60, 48, device="cuda")
        left = ((fckl.embedding(W.detach() + D, tokens, 3.0) - y.detach()).double() * g.double()).sum()
        right = (D.double() * dW.double()).sum()
        assert abs(left - right) <= 1e-5 * (D.double() * dW.double()).abs().sum()


@gpu
def test_streams_and_workspaces(fckl):
    """On another stream, with a workspace of the caller's, twice at once, and captured and replayed."""
    W, g = rows(500, 64, "bf16", 1).contiguous(), rows(3000, 64, "bf16", 2).contiguous()
    tokens = draw_tokens(3000, 500, 3)
    y, dW = fckl.embedding(W, tokens), fckl.embedding_backward(g, tokens, 500)
    s, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    s2.wait_stream(torch.cuda.current_stream())
    ws = fckl.Workspace(3000, 64, 500, 0, 0, kind="embedding_backward")
    a = [(fckl.embedding(W, tokens, stream=st), fckl.embedding_backward(g, tokens, 500, stream=st)) for st in (s, s2) * 3]
    b = fckl.embedding_backward(g, tokens, 500, ws=ws, stream=s)
    torch.cuda.synchronize()
    assert fckl.check(ws) == fckl.OK
    assert all(torch.equal(y, p) and torch.equal(dW, q) for p, q in a) and torch.equal(b, dW)
    graph = torch.cuda.CUDAGraph()
    out, acc = torch.empty_like(y), torch.zeros_like(dW)
    with torch.cuda.graph(graph):
        fckl.embedding(W, tokens, out=out)
        fckl.embedding_backward(g, tokens, 500, dW=acc, accumulate=True)
    tokens2 = draw_tokens(3000, 500, 9)
    tokens.copy_(tokens2)
    acc.zero_()
    graph.replay()
    graph.replay()
    assert torch.equal(out, fckl.embedding(W, tokens2))
    once = fckl.embedding_backward(g, tokens2, 500)
    twice = fckl.embedding_backward(g, tokens2, 500, dW=once.clone(), accumulate=True)
    assert torch.equal(acc, twice)


# ------------------------------------------------------------------ refusals (CPU)
def test_argument_errors_launch_nothing(fckl):
    lib = fckl.load()
    before = lib.fckl_launch_count()
    p, z = ctypes.c_void_p(4096), ctypes.c_void_p(0)

    def fwd(W=p, dt=0, ldw=64, t=p, N=4, d=64, V=100, out=p, ldo=64, ws=p, n=256):
        return lib.fckl_embedding(W, dt, ldw, t, N, d, V, 1.0, out, ldo, ws, n, z)

    odd = ctypes.c_void_p(4097)
    for bad in (dict(N=-1), dict(d=0), dict(V=0), dict(ldw=63), dict(ldo=63), dict(dt=3), dict(dt=-1), dict(W=z), dict(W=odd),
                dict(t=z), dict(t=odd), dict(out=z), dict(out=odd), dict(ws=z), dict(ws=ctypes.c_void_p(128)),
                dict(dt=1, W=ctypes.c_void_p(4098))):
        assert fwd(**bad) == fckl.ERR_ARG, bad
    for bad in (dict(N=(1 << 30) + 1), dict(V=(1 << 30) + 1), dict(d=(1 << 20) + 1, ldw=1 << 21, ldo=1 << 21),
                dict(ldw=(1 << 40) + 1)):
        assert fwd(**bad) == fckl.ERR_UNSUPPORTED, bad
    assert fwd(n=255) == fckl.ERR_WORKSPACE
    assert fwd(N=0, W=z, t=z, out=z) == fckl.OK
    size = lib.fckl_embedding_backward_workspace_bytes

    def bwd(g=p, dt=0, ldg=64, t=p, N=4, d=64, V=100, dW=p, odt=1, ws=p, n=None):
        return lib.fckl_embedding_backward(g, dt, ldg, t, N, d, V, 1.0, dW, odt, 0, ws, size(4, 64, 100) if n is None else n,
                                           z)

    for bad in (dict(N=-1), dict(d=0), dict(V=0), dict(ldg=63), dict(dt=3), dict(odt=2), dict(dt=1, odt=0), dict(g=z),
                dict(g=odd), dict(t=z), dict(dW=z), dict(dW=ctypes.c_void_p(4098)), dict(ws=z),
                dict(ws=ctypes.c_void_p(128))):
        assert bwd(**bad) == fckl.ERR_ARG, bad
    assert bwd(N=(1 << 30) + 1) == fckl.ERR_UNSUPPORTED
    assert bwd(n=size(4, 64, 100) - 1) == fckl.ERR_WORKSPACE
    assert lib.fckl_launch_count() == before
    # room for the ordered positions, twice, and for two partial rows per tile of at least 8
    assert size(0, 64, 100) > 0 and size(-1, 64, 100) == 0 and size(4, 0, 100) == 0 and size((1 << 30) + 1, 64, 100) == 0
    for N, d in ((1, 1), (1000, 64), (300000, 33)):
        assert 16 * N <= size(N, d, 5000) <= 16 * N + (N // 8 + 1) * 2 * (d + 8) * 4 + 4096
    ws = fckl.Workspace(1000, 64, 5000, 0, 0, device="cpu", kind="embedding_backward")
    assert ws.nbytes == size(1000, 64, 5000)


@pytest.mark.parametrize("bad", [
    lambda f, W, t: f.embedding(W, t), lambda f, W, t: f.embedding(W.double(), t), lambda f, W, t: f.embedding(W, t.long()),
    lambda f, W, t: f.embedding(W[0], t), lambda f, W, t: f.embedding(W.t(), t),
    lambda f, W, t: f.embedding(W[:1].expand(6, 8), t), lambda f, W, t: f.embedding(W, t.view(2, 2).t()),
    lambda f, W, t: f.embedding(W, t, out=W), lambda f, W, t: f.embedding(W, t, out=W[:4].bfloat16()),
    lambda f, W, t: f.embedding_backward(W, t, 6), lambda f, W, t: f.embedding_backward(W[:4], t, 6),
    lambda f, W, t: f.embedding_backward(W[:4], t.long(), 6), lambda f, W, t: f.embedding_backward(W[:4].double(), t, 6),
    lambda f, W, t: f.embedding_backward(W[:4], t, 6, accumulate=True),
    lambda f, W, t: f.embedding_backward(W[:4], t, 6, dtype=torch.bfloat16),
    lambda f, W, t: f.embedding_backward(W[:4], t, 6, dW=W[:5]),
    lambda f, W, t: f.embedding_backward(W[:4], t, 6, dW=W, dtype=torch.float16),
    lambda f, W, t: f.embedding_backward(W[:4, :1].expand(4, 8), t, 6), lambda f, W, t: f.embedding_backward(W[0, 0], t, 6),
])
def test_binding_refusals(fckl, bad):
    """Wrong types, shapes and layouts, and tensors that are not on the GPU."""
    with pytest.raises((TypeError, ValueError)):
        bad(fckl, torch.zeros(6, 8), torch.zeros(4, dtype=torch.int32))


# ------------------------------------------------------------------ the oracle (CPU)
def test_oracle_against_matrix_products():
    rng = np.random.default_rng(0)
    W, t = rng.normal(size=(7, 3)), np.array([2, -1, 6, 2])
    hot = np.zeros((4, 7))
    hot[[0, 2, 3], [2, 6, 2]] = 1
    np.testing.assert_allclose(orc.embedding(W, t, 1.5), 1.5 * hot @ W)
    g = rng.normal(size=(4, 3))
    dW, size, count = orc.embedding_gradient(g, t, 7, 1.5, old=W)
    np.testing.assert_allclose(dW, W + 1.5 * hot.T @ g)
    np.testing.assert_allclose(size, hot.T @ np.abs(g))
    assert count.tolist() == [0, 0, 2, 0, 0, 0, 1]
