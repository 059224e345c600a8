"""Logits adjusted by rules (adjust_logits, adjust_logits_backward) against the fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24): the penalty of a repeated token is one product or quotient,
the count's product and the two subtractions and the addition of the biases' sum (B additions) are each
off by u of a value that is at most M, the largest size that any of them takes; so (5 + B) u M, and half a
step of the logits' type (at least half its smallest subnormal) for the rounding. The gradient is one
quotient or product: u and half a step. Places that no rule touches keep their bits.
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


def host(t):
    return None if t is None else t.cpu().numpy()


def half_step(want, dtype):
    info = torch.finfo(dtype)
    size = np.where(np.isfinite(want), np.abs(want), 0.0)
    return np.maximum(size * info.eps / 2, info.smallest_normal * info.eps / 2)


def close(got, want, tol):
    with np.errstate(invalid="ignore"):
        bad = ~((np.abs(got - want) <= tol) | (got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


def place(x, pad=0, offset=0, fill=float("nan")):
    """On the GPU as a view with `pad` columns of `fill` between rows and `offset` elements before."""
    N, V = x.shape
    buf = torch.full((offset + N * (V + pad) + 8,), fill, dtype=x.dtype, device="cuda")
    view = buf[offset:offset + N * (V + pad)].view(N, V + pad)[:, :V]
    view.copy_(x)
    return view


def logits(N, V, dtype, seed, pad=0, offset=0):
    return place(torch.from_numpy(np.random.default_rng(seed).normal(size=(N, V)) * 3).to(DT[dtype]), pad, offset)


def pack(keep):
    """Bits of a truth table [N, V]."""
    N, V = keep.shape
    words = np.zeros((N, -(-V // 32)), dtype=np.uint32)
    for v in range(V):
        words[:, v // 32] |= keep[:, v].astype(np.uint32) << np.uint32(v % 32)
    return torch.from_numpy(words.view(np.int32)).cuda()


def rules(N, V, L, B, seed, allowed=None, tensors=True):
    """Keyword arguments of adjust_logits. Frequent tokens in the history, some slots empty; the first of
    several rows has no history, the second allows nothing."""
    rng = np.random.default_rng(seed)
    k = {}
    if L:
        t = np.minimum((np.exp(rng.random((N, L)) * np.log(V + 1)) - 1).astype(np.int64), V - 1)
        t[rng.random((N, L)) < 0.05] = -1
        t[:, -1] = V - 1
        k["history"] = torch.from_numpy(t.astype(np.int32)).cuda()
        lengths = rng.integers(0, L + 1, N)
        lengths[0], lengths[-1] = (0, L) if N > 1 else (L, L)
        k["lengths"] = torch.from_numpy(lengths.astype(np.int32)).cuda()
        k["prompt"] = torch.from_numpy((lengths * rng.random(N)).astype(np.int32)).cuda()
    if tensors:
        k["repetition"] = torch.from_numpy(rng.uniform(0.7, 1.5, N).astype(np.float32)).cuda()
        k["frequency"] = torch.from_numpy(rng.normal(size=N).astype(np.float32)).cuda()
        k["presence"] = torch.from_numpy(rng.normal(size=N).astype(np.float32)).cuda()
    else:
        k.update(repetition=1.25, frequency=0.3, presence=0.75)
    if B:
        b = rng.integers(-1, min(V, 3 * B), size=(N, B))  # repeats among them
        b[:, 0] = V - 1
        k["bias_tokens"] = torch.from_numpy(b.astype(np.int32)).cuda()
        k["bias"] = torch.from_numpy(rng.normal(size=(N, B)).astype(np.float32) * 2).cuda()
    if allowed is not None:
        keep = rng.random((N, V)) < allowed
        if N > 1:
            keep[1] = False
        k["allowed"] = pack(keep)
    return k


def oracle(z, k):
    return orc.adjust(f64(z), *(host(k.get(n)) for n in ("history", "lengths", "prompt")),
                      *(f64(k[n]) if isinstance(k.get(n), torch.Tensor) else float(np.float32(k.get(n, d)))
                        for n, d in (("repetition", 1.0), ("frequency", 0.0), ("presence", 0.0))),
                      host(k.get("bias_tokens")), host(k.get("bias")), host(k.get("allowed")))


def check_adjust(fckl, z, k, got=None, before=None):
    before = z.clone() if before is None else before
    got = fckl.adjust_logits(z, **k) if got is None else got
    assert fckl.check() == fckl.OK
    want, size = oracle(before, k)
    B = k["bias"].shape[1] if "bias" in k else 0
    close(f64(got), want, (5 + B) * U * size * 1.001 + half_step(want, z.dtype))
    return got


def check_gradient(fckl, g, z, k, got=None):
    kk = {n: k[n] for n in ("history", "lengths", "repetition", "allowed") if n in k}
    got = fckl.adjust_logits_backward(g, z, **kk) if got is None else got
    assert fckl.check() == fckl.OK
    r = k.get("repetition", 1.0)
    want = orc.adjust_gradient(f64(g), f64(z), host(k.get("history")), host(k.get("lengths")),
                               f64(r) if isinstance(r, torch.Tensor) else float(np.float32(r)), host(k.get("allowed")))
    close(f64(got), want, U * np.abs(want) + half_step(want, z.dtype))
    return got


SIZES = [(1, 1, 1, 1), (1, 1, 0, 0), (3, 2, 5, 2), (2, 31, 7, 0), (2, 32, 7, 3), (2, 33, 70, 3), (4, 1000, 0, 40),
         (5, 1003, 300, 0), (1, 50001, 2000, 300), (3, 40007, 700, 17), (160, 2501, 33, 5), (2, 16384, 100, 1024),
         (2, 16392, 9, 4), (600, 257, 12, 2), (1, 201088, 5000, 8)]


@gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("N,V,L,B", SIZES)
def test_adjust(fckl, dtype, N, V, L, B):
    z = logits(N, V, dtype, N + V)
    for allowed in (None, 0.02, 0.97):
        k = rules(N, V, L, B, V + L, allowed, tensors=allowed != 0.02)
        before = z.clone()
        got = check_adjust(fckl, z, k)
        assert torch.equal(z, before)  # a new tensor: the logits stay
        own = z.clone()
        assert fckl.adjust_logits(own, out=own, **k) is own
        assert torch.equal(own, got)


@gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("N,V,L,B", SIZES)
def test_gradient(fckl, dtype, N, V, L, B):
    z, g = logits(N, V, dtype, N + V), logits(N, V, dtype, N + V + 1)
    for allowed in (None, 0.02, 0.97):
        k = rules(N, V, L, 0, V + L, allowed, tensors=allowed != 0.02)
        got = check_gradient(fckl, g, z, k)
        kk = {n: k[n] for n in ("history", "lengths", "repetition", "allowed") if n in k}
        own, zz = g.clone(), z.clone()
        assert fckl.adjust_logits_backward(own, z, out=own, **kk) is own and torch.equal(own, got)
        assert fckl.adjust_logits_backward(g, zz, out=zz, **kk) is zz and torch.equal(zz, got)
        one = z.clone()  # all three the same tensor
        assert torch.equal(fckl.adjust_logits_backward(one, one, out=one, **kk), fckl.adjust_logits_backward(z, z, **kk))


@gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 5), (8, 8), (13, 2)])
def test_strides_and_alignment(fckl, dtype, pad, offset):
    """Rows of the logits, the result and the history apart and off the 16-byte boundary; NaN between the
    rows is not read, and what lies there not written."""
    N, V = 6, 3001
    z, g = logits(N, V, dtype, 1, pad, offset), logits(N, V, dtype, 2, offset, pad)
    k = rules(N, V, 90, 6, 3, 0.9)
    h = torch.full((N, 100), V, dtype=torch.int32, device="cuda")  # out of range beyond L
    h[:, 4:94] = k["history"]
    want, dwant = check_adjust(fckl, z, k), check_gradient(fckl, g, z, k)
    k["history"] = h[:, 4:94]
    wide = torch.zeros(N, k["allowed"].shape[1] + 3, dtype=torch.int32, device="cuda")
    wide[:, :-3] = k["allowed"]
    k["allowed"] = wide[:, :-3]
    kk = {n: k[n] for n in ("history", "lengths", "repetition", "allowed")}
    for opad, ooff in ((0, 0), (pad, offset), (2, 3)):
        out = place(torch.zeros(N, V, dtype=DT[dtype]), opad, ooff, 7.0)
        assert torch.equal(fckl.adjust_logits(z, out=out, **k), want)
        assert torch.equal(fckl.adjust_logits_backward(g, z, out=out, **kk), dwant)
        base = out._base if out._base is not None else out
        out.fill_(7.0)
        assert (base == 7.0).all()
    own = logits(N, V, dtype, 1, pad, offset)
    assert torch.equal(fckl.adjust_logits(own, out=own, **k), want)


@gpu
@pytest.mark.parametrize("dtype", list(DT))
def test_untouched_places_keep_their_bits(fckl, dtype):
    """Without rules, and beside them: NaN, infinities, zeros of both signs, subnormals."""
    info = torch.finfo(DT[dtype])
    odd = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, info.max, info.min, info.smallest_normal,
                        info.smallest_normal * info.eps], dtype=DT[dtype], device="cuda")
    z = odd.repeat(3, 200)
    bits = torch.int32 if dtype == "fp32" else torch.int16
    assert torch.equal(fckl.adjust_logits(z).view(bits), z.view(bits))
    assert torch.equal(fckl.adjust_logits_backward(z, z).view(bits), z.view(bits))
    h = torch.tensor([[5], [700], [1799]], dtype=torch.int32, device="cuda")
    got = fckl.adjust_logits(z, h, repetition=2.0, frequency=1.0)
    same = torch.ones_like(z, dtype=torch.bool).scatter_(1, h.long(), False)
    assert torch.equal(got[same].view(bits), z[same].view(bits))
    keep = torch.zeros(3, 1800, dtype=torch.bool)
    keep[:, ::2] = True
    m = pack(keep.numpy())
    got = fckl.adjust_logits(z, allowed=m)
    keep = keep.cuda()
    assert torch.equal(got[keep].view(bits), z[keep].view(bits)) and (got[~keep] == -float("inf")).all()
    got = fckl.adjust_logits_backward(z, z, allowed=m)
    assert torch.equal(got[keep].view(bits), z[keep].view(bits)) and (got[~keep] == 0).all()


@gpu
@pytest.mark.parametrize("dtype", list(DT))
def test_extreme_logits_under_penalties(fckl, dtype):
    """Infinities, NaN, zeros and the type's largest numbers under each rule: the fp32 arithmetic, rounded."""
    info = torch.finfo(DT[dtype])
    z = torch.tensor([[float("nan"), float("inf"), -float("inf"), 0.0, -0.0, info.max, info.min, info.smallest_normal]],
                     dtype=DT[dtype], device="cuda").repeat(1, 3)
    h = torch.arange(24, dtype=torch.int32, device="cuda").view(1, 24)
    x = z.cpu().float()
    for r in (0.5, 2.0):
        want = torch.where(x > 0, x / r, x * r)
        got = fckl.adjust_logits(z, h, repetition=r).cpu()
        assert torch.equal(got.nan_to_num(nan=5.0), want.to(z.dtype).nan_to_num(nan=5.0))
        got = fckl.adjust_logits(z, h, repetition=r, frequency=2.0, presence=0.5).cpu()
        assert torch.equal(got.nan_to_num(nan=5.0), (want - 2.0 - 0.5).to(z.dtype).nan_to_num(nan=5.0))
        g = torch.ones_like(z)
        slope = torch.where(x > 0, torch.tensor(1 / r), torch.tensor(r))
        assert torch.equal(fckl.adjust_logits_backward(g, z, h, repetition=r).cpu(), slope.to(z.dtype))
    ban = torch.tensor([[3, 5]], dtype=torch.int32, device="cuda")
    got = fckl.adjust_logits(z, bias_tokens=ban, bias=torch.tensor([[-float("inf"), 1.0]], device="cuda"))
    assert got[0, 3] == -float("inf") and got[0, 4] == 0


@gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("N,V,L,B", [(2, 40007, 20000, 30), (3, 300, 16000, 5), (40, 9001, 13000, 2), (2, 5001, 12280, 8),
                                     (1, 90001, 12300, 1024)])
def test_long_histories(fckl, dtype, N, V, L, B):
    """Histories on both sides of what the table of touched tokens takes, into a tensor, in place and off the
    vectors' boundaries, and the gradient."""
    z, g = logits(N, V, dtype, N + V), logits(N, V, dtype, N + V + 1)
    for allowed in (None, 0.9):
        k = rules(N, V, L, B, V + L, allowed)
        got = check_adjust(fckl, z, k)
        own = z.clone()
        assert torch.equal(fckl.adjust_logits(own, out=own, **k), got)
        off = place(torch.zeros(N, V, dtype=DT[dtype]), 3, 1, 7.0)
        assert torch.equal(fckl.adjust_logits(z, out=off, **k), got)
        d = check_gradient(fckl, g, z, k)
        kk = {n: k[n] for n in ("history", "lengths", "repetition", "allowed") if n in k}
        own = g.clone()
        assert torch.equal(fckl.adjust_logits_backward(own, z, out=own, **kk), d)
        only = {n: k[n] for n in kk if n != "repetition"}
        got = check_adjust(fckl, z, dict(only, repetition=1.5))
        own = z.clone()
        assert torch.equal(fckl.adjust_logits(own, out=own, repetition=1.5, **only), got)


@gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("N,V,L,B", [(1, 201088, 8192, 100), (16, 201088, 8192, 100), (2, 182000, 8000, 300), (2, 210000, 8000, 0),
                                     (1, 112000, 8000, 1024), (2, 128256, 8000, 860)])
def test_long_histories_that_fill_shared_memory(fckl, dtype, N, V, L, B):
    """The largest table of touched tokens, its bits and biases at the size where, with every stage, they just
    fill a block's shared memory in one segment: into a new tensor, and in place with and without a mask."""
    z = logits(N, V, dtype, N + V)
    for allowed in (None, 0.9):
        k = rules(N, V, L, B, V + L, allowed)
        got = check_adjust(fckl, z, k)
        own = z.clone()
        assert torch.equal(fckl.adjust_logits(own, out=own, **k), got)


@gpu
def test_biases_of_one_token(fckl):
    """A token's several biases are added in their order: all slots one token, and pairs far apart."""
    z = logits(2, 3000, "fp32", 1)
    b = torch.randn(2, 1024, device="cuda")
    t = torch.full((2, 1024), 2999, dtype=torch.int32, device="cuda")
    t[1] = torch.arange(1024, device="cuda").remainder(512).int()
    got = fckl.adjust_logits(z, bias_tokens=t, bias=b)
    want = z.clone()
    total = np.float32(0)
    for x in b[0].cpu().numpy():
        total = np.float32(total + x)
    want[0, 2999] += float(total)
    want[1, :512] += b[1, :512] + b[1, 512:]
    assert torch.equal(got, want)
    own = z.clone()
    assert torch.equal(fckl.adjust_logits(own, bias_tokens=t, bias=b, out=own), want)


@gpu
def test_histories_that_meet_the_limits(fckl):
    """Lengths and prompts outside the row are held to it; a token repeated throughout; a long history."""
    N, V, L = 4, 300, 65
    z = logits(N, V, "fp32", 1)
    h = torch.full((N, L), 17, dtype=torch.int32, device="cuda")
    lengths = torch.tensor([-5, 0, 1 << 30, L], dtype=torch.int32, device="cuda")
    prompt = torch.tensor([0, 3, -7, 1 << 30], dtype=torch.int32, device="cuda")
    k = dict(history=h, lengths=lengths, prompt=prompt, repetition=1.5, frequency=0.25, presence=1.0)
    got = check_adjust(fckl, z, k)
    assert torch.equal(got[:2], z[:2])
    assert abs(float(got[2, 17]) - (float(z[2, 17]) * (1.5 if z[2, 17] <= 0 else 1 / 1.5) - 0.25 * L - 1.0)) < 1e-5
    long = torch.full((1, 1048575), 299, dtype=torch.int32, device="cuda")
    got = fckl.adjust_logits(z[:1], long, frequency=0.5)
    assert float(got[0, 299]) == float(np.float32(f64(z)[0, 299] - 0.5 * 1048575)) and torch.equal(got[0, :299], z[0, :299])
    assert fckl.check() == fckl.OK
    with pytest.raises(fckl.FcklError):
        fckl.adjust_logits(z[:1], torch.zeros(1, 1048576, dtype=torch.int32, device="cuda"))


@gpu
def test_shared_rules(fckl):
    """One row of allowed tokens for all, given once or expanded; numbers against tensors that hold them."""
    z = logits(5, 1001, "bf16", 1)
    k = rules(5, 1001, 40, 3, 2, tensors=False)
    m = pack((np.random.default_rng(0).random((1, 1001)) < 0.5))
    a = check_adjust(fckl, z, dict(k, allowed=m[0]))
    assert torch.equal(fckl.adjust_logits(z, **dict(k, allowed=m.expand(5, -1))), a)
    assert torch.equal(fckl.adjust_logits(z, **dict(k, allowed=m.repeat(5, 1))), a)
    for n in ("repetition", "frequency", "presence"):
        k[n] = torch.full((5,), k[n], device="cuda")
    assert torch.equal(fckl.adjust_logits(z, **dict(k, allowed=m[0])), a)


@gpu
def test_bad_ids_are_reported_and_skipped(fckl):
    z = logits(2, 100, "fp16", 1)
    want = fckl.adjust_logits(z, torch.tensor([[3, -1], [4, -1]], dtype=torch.int32, device="cuda"), repetition=2.0)
    assert fckl.check() == fckl.OK
    for bad in (100, -2, 2 ** 31 - 1, -2 ** 31):
        h = torch.tensor([[3, bad], [4, -1]], dtype=torch.int32, device="cuda")
        assert torch.equal(fckl.adjust_logits(z, h, repetition=2.0), want)
        assert fckl.check(raise_on_error=False) == fckl.ERR_INDEX
        b = torch.tensor([[bad], [-1]], dtype=torch.int32, device="cuda")
        assert torch.equal(fckl.adjust_logits(z, bias_tokens=b, bias=torch.ones(2, 1, device="cuda")), z)
        assert fckl.check(raise_on_error=False) == fckl.ERR_INDEX
        fckl.adjust_logits_backward(z, z, h, repetition=2.0)
        assert fckl.check(raise_on_error=False) == fckl.ERR_INDEX
    assert fckl.adjust_logits(z[:0], h[:0]).shape == (0, 100) and fckl.check() == fckl.OK


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_autograd_and_differences(fckl, dtype):
    """The gradient through autograd is the direct call's, also of a broadcast upstream gradient; in fp32
    it agrees with differences of the adjusted logits (piecewise linear in z: exact but for rounding)."""
    N, V = 3, 403
    z = logits(N, V, dtype, 4).contiguous()
    k = rules(N, V, 60, 4, 5, 0.6)
    leaf = z.clone().requires_grad_()
    y = fckl.differentiable_adjusted_logits(leaf, **k)
    assert torch.equal(y, fckl.adjust_logits(z, **k))
    keep = torch.isfinite(y)
    g = logits(N, V, dtype, 6).contiguous()
    d, = torch.autograd.grad(y, leaf, g, retain_graph=True)
    check_gradient(fckl, g, z, k, got=d)
    one, = torch.autograd.grad(y, leaf, torch.ones((), dtype=y.dtype, device="cuda").expand_as(y))
    check_gradient(fckl, torch.ones_like(g), z, k, got=one)
    number = dict(k, repetition=1.5)
    y2 = fckl.differentiable_adjusted_logits(leaf, **number)
    check_gradient(fckl, g, z, number, got=torch.autograd.grad(y2, leaf, g)[0])
    if dtype == "fp32":
        e = 2.0 ** -4  # away from the bend at z = 0
        far = (z.abs() > 2 * e) & keep
        diff = (fckl.adjust_logits(z + e, **k) - fckl.adjust_logits(z - e, **k)) / (2 * e)
        assert ((diff - one).abs()[far] <= 64 * U / e * 8).all()


@gpu
def test_streams_and_graphs(fckl):
    z = logits(20, 5001, "bf16", 1).contiguous()
    k = rules(20, 5001, 200, 9, 2, 0.5)
    kk = {n: k[n] for n in ("history", "lengths", "repetition", "allowed")}
    want, dwant = fckl.adjust_logits(z, **k), fckl.adjust_logits_backward(z, z, **kk)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, dgot = fckl.adjust_logits(z, stream=s, **k), fckl.adjust_logits_backward(z, z, stream=s, **kk)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(dgot, dwant)
    out, graph = torch.empty_like(z), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out.copy_(z)
        fckl.adjust_logits(out, out=out, **k)
    k["history"].copy_(k["history"].flip(0))
    z.mul_(0.5)
    graph.replay()
    assert torch.equal(out, fckl.adjust_logits(z, **k))


@gpu
def test_offsets_past_32_bits(fckl):
    """More than 2^31 logits: the last rows match the same rows on their own, bit for bit."""
    N, V = 70000, 32000
    z = torch.empty(N, V, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    h = torch.randint(0, V, (N, 20), device="cuda", dtype=torch.int32)
    m = torch.randint(-2 ** 31, 2 ** 31, (N, 1000), device="cuda", dtype=torch.int64).int()
    tail = slice(N - 50, N)
    own = fckl.adjust_logits(z[tail].clone(), h[tail].contiguous(), repetition=1.5, frequency=0.5, allowed=m[tail].contiguous())
    got = fckl.adjust_logits(z, h, repetition=1.5, frequency=0.5, allowed=m)
    assert torch.equal(got[tail], own)
    check_adjust(fckl, z[tail], dict(history=h[tail], repetition=1.5, frequency=0.5, allowed=m[tail]), got=own)
    d = fckl.adjust_logits_backward(z, z, h, repetition=1.5, allowed=m)
    assert torch.equal(d[tail], fckl.adjust_logits_backward(z[tail].clone(), z[tail].clone(), h[tail].contiguous(),
                                                           repetition=1.5, allowed=m[tail].contiguous()))


# ------------------------------------------------------------------ refusals (CPU)
def test_argument_errors_launch_nothing(fckl):
    lib = fckl.load()
    before = lib.fckl_launch_count()
    p, z, odd = ctypes.c_void_p(4096), ctypes.c_void_p(0), ctypes.c_void_p(4097)

    def fwd(x=p, dt=0, ld=100, N=4, V=100, h=p, ldh=9, L=9, n=p, m=p, r=z, r1=1.0, f=z, pr=z, bt=p, b=p, B=3, a=p, lda=4,
            out=ctypes.c_void_p(1 << 20), ldo=100, ws=p, nb=256):
        return lib.fckl_adjust_logits(x, dt, ld, N, V, h, ldh, L, n, m, r, r1, f, 0.0, pr, 0.0, bt, b, B, a, lda, out, ldo,
                                      ws, nb, z)

    nan = float("nan")
    for bad in (dict(N=-1), dict(V=0), dict(L=-1), dict(B=-1), dict(ld=99), dict(ldo=99), dict(ldh=8), dict(lda=3),
                dict(lda=-1), dict(dt=3), dict(dt=-1), dict(x=z), dict(x=odd), dict(out=z), dict(out=odd), dict(h=z),
                dict(h=odd), dict(n=odd), dict(m=odd), dict(r=odd), dict(f=odd), dict(pr=odd), dict(bt=z), dict(b=z),
                dict(bt=odd), dict(b=odd), dict(a=odd), dict(r1=0.0), dict(r1=-1.0), dict(r1=nan), dict(out=p, ldo=101),
                dict(ws=z), dict(ws=ctypes.c_void_p(128))):
        assert fwd(**bad) == fckl.ERR_ARG, bad
    for bad in (dict(V=(1 << 30) + 1, ld=1 << 31, ldo=1 << 31), dict(N=(1 << 40) + 1), dict(L=1 << 20, ldh=1 << 20),
                dict(B=1025), dict(ld=(1 << 40) + 1), dict(ldh=(1 << 40) + 1)):
        assert fwd(**bad) == fckl.ERR_UNSUPPORTED, bad
    assert fwd(nb=255) == fckl.ERR_WORKSPACE
    assert fwd(N=0, x=z, out=z, h=z) == fckl.OK

    def bwd(g=p, dt=0, ldg=100, x=p, ld=100, N=4, V=100, h=p, ldh=9, L=9, n=p, r=z, r1=1.0, a=p, lda=4,
            out=ctypes.c_void_p(1 << 20), ldo=100, ws=p, nb=256):
        return lib.fckl_adjust_logits_backward(g, dt, ldg, x, ld, N, V, h, ldh, L, n, r, r1, a, lda, out, ldo, ws, nb, z)

    for bad in (dict(ldg=99), dict(ld=99), dict(ldo=99), dict(g=z), dict(g=odd), dict(x=z), dict(x=odd), dict(h=z),
                dict(r1=0.0), dict(dt=7), dict(out=p, ldo=101), dict(g=ctypes.c_void_p(8192), out=p, ldo=101)):
        assert bwd(**bad) == fckl.ERR_ARG, bad
    assert bwd(nb=0) == fckl.ERR_WORKSPACE and bwd(N=0) == fckl.OK
    assert lib.fckl_launch_count() == before


@pytest.mark.parametrize("bad", [
    lambda f, z, h: f.adjust_logits(z, h), lambda f, z, h: f.adjust_logits(z.double(), h),
    lambda f, z, h: f.adjust_logits(z[0], h), lambda f, z, h: f.adjust_logits(z, h.long()),
    lambda f, z, h: f.adjust_logits(z, h[:2]), lambda f, z, h: f.adjust_logits(z, lengths=h[:, 0].contiguous()),
    lambda f, z, h: f.adjust_logits(z, h, lengths=h[:, 0]), lambda f, z, h: f.adjust_logits(z, h, repetition=0.0),
    lambda f, z, h: f.adjust_logits(z, h, repetition=torch.ones(2)), lambda f, z, h: f.adjust_logits(z, bias=z),
    lambda f, z, h: f.adjust_logits(z, bias_tokens=h, bias=torch.zeros(3, 3)),
    lambda f, z, h: f.adjust_logits(z, allowed=torch.zeros(3, 2, dtype=torch.int32)),
    lambda f, z, h: f.adjust_logits(z, allowed=torch.zeros(3, 1, dtype=torch.bool)),
    lambda f, z, h: f.adjust_logits(z, h, out=z[:2]), lambda f, z, h: f.adjust_logits(z[:1].expand(3, 8), h),
    lambda f, z, h: f.adjust_logits(z, h[:1].expand(3, 2)),
    lambda f, z, h: f.adjust_logits_backward(z, z, h), lambda f, z, h: f.adjust_logits_backward(z[:2], z, h),
    lambda f, z, h: f.adjust_logits_backward(z.half(), z, h),
])
def test_binding_refusals(fckl, bad):
    """Wrong types, shapes and layouts, and tensors that are not on the GPU."""
    with pytest.raises((TypeError, ValueError)):
        bad(fckl, torch.zeros(3, 8), torch.zeros(3, 2, dtype=torch.int32))


@pytest.mark.parametrize("name", ["repetition", "frequency", "presence", "bias"])
def test_penalties_that_require_a_gradient_are_refused(fckl, name):
    """The rules have a gradient of the logits alone: none is dropped without notice. Without gradients, and
    for tensors that ask for none, that check does not apply (and the CPU tensors are refused for where they are)."""
    z, h = torch.zeros(3, 8, requires_grad=True), torch.zeros(3, 2, dtype=torch.int32)
    k = dict(history=h, repetition=torch.ones(3), frequency=torch.ones(3), presence=torch.ones(3), bias_tokens=h,
             bias=torch.ones(3, 2))
    k[name].requires_grad_()
    with pytest.raises(ValueError, match=f"{name} has no gradient"):
        fckl.differentiable_adjusted_logits(z, **k)
    with pytest.raises(Exception) as e, torch.no_grad():
        fckl.differentiable_adjusted_logits(z, **k)
    assert "has no gradient" not in str(e.value)
    k[name] = k[name].detach()
    with pytest.raises(Exception) as e:
        fckl.differentiable_adjusted_logits(z, **k)
    assert "has no gradient" not in str(e.value)


@gpu
def test_penalties_that_require_no_gradient_here(fckl):
    """The same tensors detached, or without gradients, give what the direct call gives."""
    z = logits(3, 40, "fp32", 1).contiguous()
    k = rules(3, 40, 9, 2, 2)
    want = fckl.adjust_logits(z, **k)
    for name in ("repetition", "frequency", "presence", "bias"):
        own = dict(k, **{name: k[name].clone().requires_grad_()})
        with pytest.raises(ValueError, match=f"{name} has no gradient"):
            fckl.differentiable_adjusted_logits(z, **own)
        with torch.no_grad():
            assert torch.equal(fckl.differentiable_adjusted_logits(z, **own), want)
        own[name] = own[name].detach()
        assert torch.equal(fckl.differentiable_adjusted_logits(z.clone().requires_grad_(), **own), want)


# ------------------------------------------------------------------ the oracle (CPU)
def test_oracle_closed_forms():
    z = np.array([[2.0, -2.0, 1.0, 0.5, 4.0]])
    h = np.array([[0, 1, 0, 1, -1, 3]])
    out, _ = orc.adjust(z, h, np.array([5]), np.array([2]), 2.0, 0.25, 0.5, np.array([[2, 2, -1]]),
                        np.array([[1.0, 2.0, 9.0]]), np.array([[0b01111]]))
    np.testing.assert_allclose(out[0], [1.0 - 0.75, -4.0 - 0.75, 4.0, 0.5, -np.inf])
    g = orc.adjust_gradient(np.ones((1, 5)), z, h, np.array([5]), 2.0, np.array([0b01111]))
    np.testing.assert_allclose(g[0], [0.5, 2.0, 1.0, 1.0, 0.0])
