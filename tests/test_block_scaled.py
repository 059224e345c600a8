"""The 8-bit block-scaled projection against its fp64 restatement.

Quantisation is exact: values and scales have to be equal. The product, on the same 8-bit values
and scales (u = 2^-24): products of two e4m3 values are exact in fp32; K of them are added in fp32,
each addition truncated at worst (2u), then ceil(K / 128) scaled sums with two roundings for the
scale, one product-sum each: at most (2 K + ceil(K / 128) + 3) u sum |a b| =: e, and half a step
of a bf16 result (2^-8 relative).
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import block_scaled_oracle as orc
from oracle import fckl_oracle, scoring_oracle

gpu = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def test_oracle_values_against_torch():
    """All codes and the roundings between them, against torch's conversion."""
    v = orc.e4m3_values()
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(v, codes)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=4000) * 10.0 ** rng.uniform(-4, 2.6, 4000), (v[1:] + v[:-1]) / 2, -v,
                        [448.0, 447.9, -448.0, 0.0, 2.0 ** -10, 2.0 ** -11]]).clip(-448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(orc.round_e4m3(x), want.astype(np.float64))


def draw(R, K, dtype, seed, pad=0, offset=0):
    """x [R, K] on the GPU with blocks of very different sizes, zeros and huge values among them."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(R, K)) * 10.0 ** rng.integers(-3, 3, size=(R, 1))
    x[:, ::97] *= 30
    if R > 2:
        x[1] = 0.0
    buf = torch.full((offset + R * (K + pad) + 8,), float("nan"), dtype=DT[dtype], device="cuda")
    view = buf[offset:offset + R * (K + pad)].view(R, K + pad)[:, :K]
    view.copy_(torch.from_numpy(x).to(DT[dtype]))
    return view


def f64(t):
    return t.detach().float().cpu().double().numpy()


def same_quantisation(x, rows, q, scale):
    w_q, w_s = orc.quantize(f64(x), rows)
    assert tuple(q.shape) == tuple(x.shape) and tuple(scale.shape) == w_s.shape
    assert np.array_equal(scale.cpu().numpy(), w_s)
    assert np.array_equal(f64(q), w_q)


@gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("R,K,pad,offset", [(1, 1, 0, 0), (3, 8, 0, 0), (2, 128, 0, 0), (130, 129, 0, 0), (7, 1000, 0, 0),
                                            (128, 256, 0, 0), (257, 200, 3, 1), (33, 320, 8, 8), (5, 2880, 0, 3)])
def test_quantize(fckl, dtype, rows, R, K, pad, offset):
    x = draw(R, K, dtype, R + K, pad, offset)
    q, scale = fckl.block_quantize(x, rows=rows)
    assert q.dtype == torch.float8_e4m3fn and (R == 1 or q.stride(0) % 16 == 0)
    same_quantisation(x, rows, q, scale)


@gpu
@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_extremes(fckl, rows):
    """The smallest and largest numbers, quotients on the borders between values, NaN and inf."""
    v = orc.e4m3_values()
    x = np.zeros((6, 384), dtype=np.float32)
    x[0, :127] = v                               # amax 448: scale 1, every value itself
    x[1, :126] = (v[1:] + v[:-1]) / 2            # every border
    x[1, 127] = 448
    x[2] = 1e-45                                 # below the smallest scale
    x[3] = 3.4e38
    x[4, ::2] = -1e-30
    x[5, 128:256] = np.linspace(-7.77, 7.77, 128)
    xt = torch.from_numpy(x).cuda()
    same_quantisation(xt, rows, *fckl.block_quantize(xt, rows=rows))
    # every scale exponent the quotients' fast form takes and leaves, with odd mantissas
    rng = np.random.default_rng(3)
    x = (rng.normal(size=(254, 128)) * 2.0 ** np.arange(-127, 127)[:, None]).astype(np.float32)
    x[:, 64:] *= 1e-3
    xt = torch.from_numpy(x).cuda()
    same_quantisation(xt, rows, *fckl.block_quantize(xt, rows=rows))
    xt = torch.randn(3, 256, device="cuda")
    xt[1, 5] = float("nan")
    q, scale = fckl.block_quantize(xt, rows=1)
    nan = torch.isnan(q.float())
    assert nan[1, 5] and nan.sum() == 1 and torch.isfinite(scale).all()
    xt[2, 200] = float("inf")
    q, scale = fckl.block_quantize(xt, rows=1)
    assert torch.isinf(scale[2, 1]) and (q[2, 128:200].float() == 0).all() and torch.isnan(q[2, 200].float())


@gpu
def test_quantize_many_quotients(fckl):
    """A million quotients of fp32 values with full mantissas against the true ones in 64 bits."""
    x = torch.randn(8192, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(5)) * 3
    q, scale = fckl.block_quantize(x)
    want = (x.double() / scale.double()).float().to(torch.float8_e4m3fn)
    assert torch.equal(q.view(torch.uint8), want.view(torch.uint8))


def check_product(fckl, a, sa, b, sb, **kw):
    exact, size = orc.matmul(f64(a), sa.cpu().numpy(), f64(b), sb.cpu().numpy())
    K = a.shape[1]
    e = (2 * K + -(-K // 128) + 3) * U * size
    for dt, half in ((torch.float32, U), (torch.bfloat16, 2.0 ** -8)):
        c = fckl.block_scaled_matmul(a, sa, b, sb, out_dtype=dt, **kw)
        assert fckl.check() == fckl.OK and c.dtype == dt
        err = np.abs(f64(c) - exact)
        bad = err > e + half * (np.abs(exact) + e) + 1e-38
        assert not bad.any(), (np.argwhere(bad)[:4], err[bad][:4], e[bad][:4])
    return exact


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 128, 128), (3, 257, 130), (128, 256, 256), (129, 1000, 72),
                                   (300, 513, 2880), (16, 5000, 1024), (257, 129, 16), (1, 20001, 520)])
def test_product(fckl, M, N, K):
    a, sa = fckl.block_quantize(draw(M, K, "bf16", 1), rows=1)
    b, sb = fckl.block_quantize(draw(N, K, "bf16", 2), rows=128)
    check_product(fckl, a, sa, b, sb)


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 5000, 2880), (7, 33, 64), (8, 1000, 136), (9, 129, 8), (17, 2000, 1000),
                                   (24, 500, 384), (25, 77, 129), (32, 4099, 520), (33, 700, 256), (32, 300, 4096),
                                   (2, 300, 100000)])
def test_product_decode(fckl, M, N, K):
    """Few rows: both sides of the decoding form's limits (rows, shared memory), ragged K and N; what
    lies past K in the rows' padding, NaNs here, takes no part."""
    a, sa = fckl.block_quantize(draw(M, K, "bf16", 1), rows=1)
    b, sb = fckl.block_quantize(draw(N, K, "bf16", 2), rows=128)

    def padded(q):
        buf = torch.full((q.shape[0], -(-K // 16) * 16 + 32), 0x7F, dtype=torch.uint8, device="cuda")
        buf[:, :K] = q.view(torch.uint8)
        return buf.view(torch.float8_e4m3fn)[:, :K]

    check_product(fckl, padded(a), sa, padded(b), sb)


@gpu
def test_product_layouts(fckl):
    """Rows apart, scales in other layouts, results into rows of any alignment with nothing written
    beside them."""
    M, N, K = 70, 300, 200
    big_a = torch.zeros(M, 320, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    big_b = torch.zeros(N, 224, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    q, sa = fckl.block_quantize(draw(M, K, "fp32", 3))
    big_a[:, 16:16 + K].view(torch.uint8).copy_(q.view(torch.uint8))
    a = big_a[:, 16:16 + K]
    q, sb = fckl.block_quantize(draw(N, K, "fp32", 4), rows=128)
    big_b[:, :K].view(torch.uint8).copy_(q.view(torch.uint8))
    b = big_b[:, :K]
    sa = sa.contiguous()                                                     # by row
    wide = torch.full((3, 9), float("nan"), device="cuda")
    wide[:, 1:8:4] = sb
    sb = wide[:, 1:8:4]                                                      # every fourth column
    exact = check_product(fckl, a, sa, b, sb)
    for dt, off, pad in ((torch.bfloat16, 3, 5), (torch.float32, 1, 2), (torch.bfloat16, 8, 4)):
        buf = torch.full((off + M * (N + pad) + 9,), 77.0, dtype=dt, device="cuda")
        out = buf[off:off + M * (N + pad)].view(M, N + pad)[:, :N]
        fckl.block_scaled_matmul(a, sa, b, sb, out=out)
        fckl.check()
        assert torch.equal(out, fckl.block_scaled_matmul(a, sa, b, sb, out_dtype=dt))
        assert (buf[:off] == 77).all() and (buf[off:off + M * (N + pad)].view(M, N + pad)[:, N:] == 77).all()
        assert np.isfinite(exact).all()


@gpu
def test_product_keeps_nan_to_its_row(fckl):
    x = torch.randn(5, 300, device="cuda")
    x[2, 299] = float("nan")
    W8, ws = fckl.block_quantize(torch.randn(400, 300, device="cuda"), rows=128)
    c = fckl.block_scaled_projection(x, W8, ws)
    fckl.check()
    assert torch.isnan(c[2]).all() and torch.isfinite(c[[0, 1, 3, 4]]).all()


@gpu
def test_projection_is_its_steps_streams_graph_and_empty(fckl):
    H, W = draw(200, 256, "bf16", 5), draw(1000, 256, "bf16", 6)
    W8, sw = fckl.block_quantize(W, rows=128)
    want = fckl.block_scaled_matmul(*fckl.block_quantize(H), W8, sw)
    assert torch.equal(fckl.block_scaled_projection(H, W8, sw), want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = fckl.block_scaled_projection(H, W8, sw, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fckl.block_scaled_projection(H, W8, sw)
    H.copy_(draw(200, 256, "bf16", 7))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, fckl.block_scaled_projection(H, W8, sw)) and not torch.equal(got, want)
    assert tuple(fckl.block_scaled_projection(H[:0], W8, sw).shape) == (0, 1000)


@gpu
def test_offsets_past_32_bits(fckl):
    """More than 2^31 results: the last rows are those of the same positions on their own."""
    M, N, K = 36000, 60000, 64
    H = torch.randn(M, K, device="cuda").bfloat16()
    W8, sw = fckl.block_quantize(torch.randn(N, K, device="cuda"), rows=128)
    c = fckl.block_scaled_projection(H, W8, sw)
    fckl.check()
    assert torch.equal(c[-300:], fckl.block_scaled_projection(H[-300:].clone(), W8, sw))


@gpu
def test_teacher_cache_from_the_8_bit_head(fckl):
    """The pieces together: 8-bit logits, their top K as a teacher cache, the loss and its gradient
    against the cache; the cache is that of the same logits by the oracle."""
    N, d, V, K = 150, 256, 3000, 20
    Ht, Wt = torch.randn(N, d, device="cuda").bfloat16(), (torch.randn(V, d, device="cuda") / 16).bfloat16()
    W8, sw = fckl.block_quantize(Wt, rows=128)
    logits = fckl.block_scaled_projection(Ht, W8, sw, out_dtype=torch.float32)
    none = torch.empty(N, 0, dtype=torch.int32, device="cuda")
    _, _, _, idx, logp = fckl.token_logprobs(logits, none, top=K)
    w_idx, w_logp = scoring_oracle.alternatives(f64(logits), K)
    assert np.array_equal(idx.cpu().numpy(), w_idx) and np.abs(f64(logp) - w_logp).max() < 1e-5
    loss, _, dH, dW = fckl.forward_backward(Ht, Wt, idx, logp, 64)
    assert fckl.check() == fckl.OK
    # the loss's own tolerance (1e-3 of 1 + |loss| per position); the cache is not renormalised, so the
    # least loss of a position is S log(S / Q), the student's mass Q on those tokens, not 0
    want, _, rl = fckl_oracle.forward(f64(Ht), f64(Wt), w_idx, logp.cpu().numpy(), 64)
    assert abs(float(loss) - want) <= N * 1e-3 * (1 + np.abs(rl).max())
    assert torch.isfinite(dH).all() and torch.isfinite(dW).all()


# ------------------------------------------------------------------ refusals (CPU)
def test_argument_errors_launch_nothing(fckl):
    lib = fckl.load()
    before = lib.fckl_launch_count()
    p, z, odd = ctypes.c_void_p(256), ctypes.c_void_p(0), ctypes.c_void_p(257)

    def quant(x=p, dt=0, ldx=64, rows=4, cols=64, br=1, q=p, ldq=64, s=p, rs=1, cs=4):
        return lib.fckl_block_quantize(x, dt, ldx, rows, cols, br, q, ldq, s, rs, cs, z)

    for bad in (dict(rows=-1), dict(cols=0), dict(dt=3), dict(br=2), dict(ldx=63), dict(ldq=48), dict(rs=0),
                dict(cs=0), dict(x=z), dict(x=odd), dict(q=z), dict(q=ctypes.c_void_p(264)), dict(s=z), dict(s=odd)):
        assert quant(**bad) == fckl.ERR_ARG, bad
    for bad in (dict(ldq=72), dict(rows=(1 << 30) + 1), dict(cols=(1 << 20) + 1, ldx=1 << 21, ldq=1 << 21)):
        assert quant(**bad) == fckl.ERR_UNSUPPORTED, bad
    assert quant(rows=0, x=z, q=z, s=z) == fckl.OK

    def mm(a=p, lda=64, sa=p, sars=1, sacs=4, b=p, ldb=64, sb=p, sbrs=1, sbcs=1, M=4, N=100, K=64, c=p, dt=0, ldc=100,
           ws=p, n=256):
        return lib.fckl_block_scaled_matmul(a, lda, sa, sars, sacs, b, ldb, sb, sbrs, sbcs, M, N, K, c, dt, ldc, ws, n,
                                            z)

    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(dt=2), dict(lda=48), dict(ldb=48), dict(ldc=99), dict(sars=0),
                dict(sbcs=0), dict(a=z), dict(b=z), dict(sa=z), dict(sb=odd), dict(c=z), dict(c=odd),
                dict(a=ctypes.c_void_p(264)), dict(ws=z)):
        assert mm(**bad) == fckl.ERR_ARG, bad
    for bad in (dict(lda=72), dict(ldb=72), dict(M=(1 << 30) + 1), dict(N=(1 << 30) + 1, ldc=1 << 31),
                dict(K=(1 << 20) + 1, lda=1 << 21, ldb=1 << 21)):
        assert mm(**bad) == fckl.ERR_UNSUPPORTED, bad
    assert mm(n=128) == fckl.ERR_WORKSPACE
    assert mm(M=0, a=z, sa=z, c=z) == fckl.OK
    assert lib.fckl_launch_count() == before


@pytest.mark.parametrize("bad", [
    lambda f, x, q, s: f.block_quantize(x, rows=64), lambda f, x, q, s: f.block_quantize(x.double()),
    lambda f, x, q, s: f.block_quantize(x[0]), lambda f, x, q, s: f.block_quantize(x),
    lambda f, x, q, s: f.block_scaled_matmul(x, s, q, s), lambda f, x, q, s: f.block_scaled_matmul(q, s, q[:, :16], s),
    lambda f, x, q, s: f.block_scaled_matmul(q, s[:1], q, s), lambda f, x, q, s: f.block_scaled_matmul(q, s, q, s),
    lambda f, x, q, s: f.block_scaled_matmul(q, s.double(), q, s[:1]),
    lambda f, x, q, s: f.block_scaled_matmul(q, s, q, s[:1], out_dtype=torch.float16),
    lambda f, x, q, s: f.block_scaled_projection(x, q, s), lambda f, x, q, s: f.block_scaled_projection(x[:, :8], q, s),
    lambda f, x, q, s: f.block_scaled_projection(x, q, s[:1], out_dtype=torch.float16),
    lambda f, x, q, s: f.block_scaled_projection(x.double(), q, s[:1]),
    lambda f, x, q, s: f.block_scaled_projection(x, q, s[:1]),
    lambda f, x, q, s: f.block_scaled_matmul(q[:, :24].contiguous(), s, q[:, :24].contiguous(), s[:1]),
])
def test_binding_refusals(fckl, bad):
    x = torch.zeros(3, 32)
    with pytest.raises((TypeError, ValueError)):
        bad(fckl, x, x.to(torch.float8_e4m3fn), torch.zeros(3, 1))


@gpu
@pytest.mark.parametrize("M,N,K,decoding", [
    (15, 333, 200, True), (16, 4097, 384, True), (17, 4097, 384, False),                  # rows
    (8, 300, 9856, True), (8, 300, 9984, False), (16, 300, 3840, True), (16, 300, 3968, False),  # shared memory
])
def test_product_decode_limits(fckl, M, N, K, decoding):
    """Both sides of each limit of the decoding form, and which form ran."""
    a, sa = fckl.block_quantize(draw(M, K, "bf16", 1), rows=1)
    b, sb = fckl.block_quantize(draw(N, K, "bf16", 2), rows=128)
    fckl.profile_enable(True)
    fckl.profile_read()
    check_product(fckl, a, sa, b, sb)
    torch.cuda.synchronize()
    ran = {k for k, (_, n) in fckl.profile_read().items() if n}
    fckl.profile_enable(False)
    assert ("block_matmul_skinny" in ran) == decoding and ("block_scaled_matmul" in ran) != decoding, ran


@gpu
@pytest.mark.parametrize("rows", [1, 128])
def test_scales_are_dense(fckl, rows):
    """Scales come without padding, whatever the number of blocks in a row, and the product takes them."""
    for K in (1, 128, 129, 600, 2880):
        x = draw(130, K, "bf16", K)
        q, scale = fckl.block_quantize(x, rows=rows)
        assert scale.is_contiguous()
        same_quantisation(x, rows, q, scale)
        w, sw = fckl.block_quantize(draw(200, K, "bf16", K + 1), rows=128)
        if rows == 1:
            check_product(fckl, q, scale, w, sw)
