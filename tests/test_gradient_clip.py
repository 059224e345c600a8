"""The gradients' norm and clipping against the fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24): a thread sums 32 squares in fp32, each addition (and the
square in it) off by u of the sum, so by at most 32 u; everything beyond is fp64. The norm is half of
that off, 16 u, and u for its rounding: 17 u. The coefficient is 17 u off and rounded (18 u), the product
another u and the result half a step of its type, at least half its smallest subnormal.
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


def tensor(shape, dtype, seed, offset=0, scale=1.0):
    """A tensor whose first element lies `offset` elements into a buffer of NaN."""
    n = int(np.prod(shape))
    x = torch.from_numpy(np.random.default_rng(seed).normal(size=n) * scale).to(DT[dtype])
    buf = torch.full((offset + n + 9,), float("nan"), dtype=DT[dtype], device="cuda")
    view = buf[offset:offset + n]
    view.copy_(x)
    return view.view(shape)


def check_norm(norm, grads):
    want = orc.norm([f64(g) for g in grads])
    assert norm.shape == (1,) and norm.dtype == torch.float32
    assert abs(float(norm) - want) <= 17 * U * want, (float(norm), want)


def check_scaled(got, grads, max_norm):
    """The scaled tensors against the oracle, whose coefficient is that of the exact norm."""
    _, c, want = orc.clip([f64(g) for g in grads], float(np.float32(max_norm)))
    for x, w, g in zip(got, want, grads):
        assert x.shape == g.shape
        info = torch.finfo(x.dtype)
        tol = 19 * U * np.abs(w) + np.maximum(np.abs(w) * info.eps / 2, info.smallest_normal * info.eps / 2) * 1.001
        if c == 1.0 and x.dtype == g.dtype:
            tol = 0
        assert (np.abs(f64(x) - w) <= tol).all()


SETS = {
    "one value": [((1,), "fp32", 0)],
    "one": [((300, 77), "bf16", 0)],
    "few": [((5, 7), "fp16", 1), ((8193,), "bf16", 3), ((64, 128), "fp32", 0), ((1,), "bf16", 1), ((3,), "fp32", 1)],
    "units": [((n,), t, o) for n in (8191, 8192, 8193, 16384) for t in DT for o in (0, 1, 3)],
    "many": [((1 + 37 * i % 501, 1 + i % 13), ("bf16", "fp16", "fp32")[i % 3], i % 5) for i in range(300)],
    "empty ones": [((0,), "bf16", 0), ((7, 0), "fp32", 0), ((19,), "fp16", 0), ((0,), "fp32", 0)],
    "large": [((3001, 1003), "fp32", 1), ((2000, 2048), "bf16", 0), ((4097, 513), "fp16", 5)],
}


def make(name, scale=1.0):
    return [tensor(shape, dtype, i, offset, scale) for i, (shape, dtype, offset) in enumerate(SETS[name])]


@gpu
@pytest.mark.parametrize("name", list(SETS))
def test_norm(fckl, name):
    grads = make(name)
    check_norm(fckl.gradient_norm(grads), grads)
    assert fckl.check() == fckl.OK


@gpu
@pytest.mark.parametrize("share", [0.01, 0.5, 1.5])
@pytest.mark.parametrize("name", list(SETS))
def test_clip_in_place(fckl, name, share):
    """Below, at half and above the norm; the last leaves the gradients' bits."""
    grads = make(name)
    before = [g.clone() for g in grads]
    max_norm = share * orc.norm([f64(g) for g in grads]) + (1e-3 if share > 1 else 0)
    norm = fckl.clip_gradients(grads, max_norm)
    check_norm(norm, before)
    check_scaled(grads, before, max_norm)
    assert torch.equal(norm, fckl.gradient_norm(before))


@gpu
@pytest.mark.parametrize("share", [0.25, 2.0])
@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("name", list(SETS))
def test_clip_into_buckets(fckl, name, out, share):
    """Into consecutive pieces of one buffer, at whatever alignment that gives; inputs and what lies
    around the buffer stay as they are."""
    grads = make(name)
    before = [g.clone() for g in grads]
    sizes = [g.numel() for g in grads]
    flat = torch.full((sum(sizes) + 40,), 7.0, dtype=DT[out], device="cuda")
    to = [x.view(g.shape) for x, g in zip(flat[17:17 + sum(sizes)].split(sizes), grads)]
    max_norm = share * orc.norm([f64(g) for g in grads]) + 1e-5
    check_norm(fckl.clip_gradients(grads, max_norm, out=to), before)
    check_scaled(to, before, max_norm)
    assert (flat[:17] == 7.0).all() and (flat[17 + sum(sizes):] == 7.0).all()
    assert all(torch.equal(a, b) for a, b in zip(grads, before))


@gpu
def test_more_tensors_than_one_table(fckl):
    grads = [tensor((1 + i % 7,), "bf16" if i % 2 else "fp32", i) for i in range(2000)]
    before = [g.clone() for g in grads]
    norm = fckl.clip_gradients(grads, 3.0)
    check_norm(norm, before)
    check_scaled(grads, before, 3.0)
    assert torch.equal(norm, fckl.gradient_norm(before))


@gpu
def test_no_tensors_and_none(fckl):
    assert float(fckl.gradient_norm([])) == 0.0
    assert float(fckl.clip_gradients([], 1.0)) == 0.0
    assert float(fckl.gradient_norm([None, torch.full((4,), 2.0, device="cuda"), None])) == 4.0
    g = torch.full((4,), 2.0, device="cuda")
    assert float(fckl.clip_gradients([None, g], 0.0)) == 4.0 and (g == 0).all()
    zeros = torch.zeros(100000, device="cuda")
    assert float(fckl.clip_gradients([zeros], 1.0)) == 0.0 and (zeros == 0).all()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-18, 1e-12, 1e12, 1e19, 1e30])
def test_gradients_of_any_size(fckl, dtype, scale):
    """Squares that leave fp32's range on either side, alone and beside ordinary ones."""
    tiny = [tensor((30001,), dtype, 1, 1, scale)]
    check_norm(fckl.gradient_norm(tiny), tiny)
    mixed = tiny + [tensor((1000,), dtype, 2, 0, 1.0)]
    mixed[0][7] = 0.0
    mixed[0][9000:9500] = 1.0
    check_norm(fckl.gradient_norm(mixed), mixed)
    if scale <= 1e12:
        before = [g.clone() for g in mixed]
        fckl.clip_gradients(mixed, 1.0)
        check_scaled(mixed, before, 1.0)


@gpu
def test_norms_that_are_not_finite(fckl):
    g = [torch.ones(5000, device="cuda"), torch.ones(33, device="cuda").bfloat16()]
    g[0][4000] = float("inf")
    assert float(fckl.gradient_norm(g)) == float("inf")
    out = [torch.empty_like(x) for x in g]
    assert float(fckl.clip_gradients(g, 1.0, out=out)) == float("inf")
    assert (out[1] == 0).all() and torch.isnan(out[0][4000]) and out[0].nan_to_num().sum() == 0
    g[0][4000] = float("nan")
    assert torch.isnan(fckl.gradient_norm(g)).all()
    assert torch.isnan(fckl.clip_gradients(g, 1.0, out=out)).all()
    assert all(torch.isnan(x).all() for x in out)
    # finite values whose norm is above the largest fp32 number: inf, yet scaled by the true one
    big = [torch.full((10000,), 3e38, device="cuda")]
    assert float(fckl.clip_gradients(big, 1.0)) == float("inf")
    assert ((big[0] - 0.01).abs() <= 20 * U * 0.01).all()


@gpu
def test_memory_orders_and_scalars(fckl):
    """Transposed and permuted tensors, which are dense in another order, and a scalar."""
    a, b = torch.randn(37, 53, device="cuda").t(), torch.randn(4, 5, 6, device="cuda").permute(2, 0, 1)
    c, s = torch.randn(3, 1, 9, device="cuda").transpose(0, 1), torch.tensor(3.0, device="cuda")
    grads = [a, b, c, s]
    before = [g.clone() for g in grads]
    check_norm(fckl.clip_gradients(grads, 2.0), before)
    check_scaled(grads, before, 2.0)


@gpu
def test_deterministic_streams_and_graphs(fckl):
    grads = make("large")
    a = fckl.gradient_norm(grads)
    s, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for st in (s, s2):
        st.wait_stream(torch.cuda.current_stream())
    got = [fckl.gradient_norm(grads, stream=st) for st in (s, s2) * 4]
    torch.cuda.synchronize()
    assert all(torch.equal(a, x) for x in got)
    out = [torch.empty_like(g) for g in grads]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = fckl.clip_gradients(grads, 5.0, out=out)
    for k in range(2):
        grads[0].mul_(2.0)
        graph.replay()
        check_norm(norm, grads)
        check_scaled(out, grads, 5.0)


@gpu
def test_more_than_2_31_elements(fckl):
    g = torch.full(((1 << 31) + 12345,), 0.5, dtype=torch.bfloat16, device="cuda")
    g[-1] = 3.0
    n = fckl.clip_gradients([g], 1.0)
    want = float(np.sqrt(0.25 * ((1 << 31) + 12344) + 9.0))
    assert abs(float(n) - want) <= 17 * U * want
    c = 1.0 / (want + 1e-6)
    for at, x in ((0, 0.5), ((1 << 31) + 5, 0.5), (-1, 3.0)):
        assert abs(float(g[at]) - x * c) <= x * c * 2 ** -8


# ------------------------------------------------------------------ refusals (CPU)
def _arrays(ptrs, sizes, types):
    n = len(ptrs)
    return (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*sizes), (ctypes.c_int * n)(*types), n


def test_argument_errors_launch_nothing(fckl):
    lib = fckl.load()
    before = lib.fckl_launch_count()
    p, z = ctypes.c_void_p(4096), ctypes.c_void_p(0)
    size = lib.fckl_gradient_norm_workspace_bytes
    assert size(-1) == 0 and size((1 << 20) + 1) == 0 and 0 < size(0) <= size(1) < size(5000)

    def norm(ptrs=(4096, 1 << 20), sizes=(10, 20), types=(0, 1), norm=p, ws=p, n=None, count=None):
        a, b, c, k = _arrays(ptrs, sizes, types)
        return lib.fckl_gradient_norm(a, b, c, k if count is None else count, norm, ws, size(2) if n is None else n, z)

    for bad in (dict(count=-1), dict(sizes=(10, -1)), dict(types=(0, 3)), dict(types=(-1, 0)), dict(ptrs=(4096, 0)),
                dict(ptrs=(4097, 1 << 20)), dict(ptrs=(4096, (1 << 20) + 2)), dict(norm=z), dict(norm=ctypes.c_void_p(2)),
                dict(ws=z), dict(ws=ctypes.c_void_p(128))):
        assert norm(**bad) == fckl.ERR_ARG, bad
    assert norm(sizes=(10, 1 << 41)) == fckl.ERR_UNSUPPORTED
    assert norm(n=size(2) - 1) == fckl.ERR_WORKSPACE
    assert lib.fckl_gradient_norm(z, z, z, 1, p, p, size(1), z) == fckl.ERR_ARG
    assert lib.fckl_gradient_norm(z, z, z, (1 << 20) + 1, p, p, 1 << 40, z) == fckl.ERR_UNSUPPORTED

    def clip(ptrs=(4096, 1 << 20), sizes=(10, 20), types=(0, 1), to=(4096, 1 << 20), to_types=(0, 1), m=1.0, n=None):
        a, b, c, k = _arrays(ptrs, sizes, types)
        d, _, e, _ = _arrays(to, sizes, to_types)
        return lib.fckl_clip_gradients(a, b, c, k, m, d, e, p, p, size(2) if n is None else n, z)

    nan = float("nan")
    for bad in (dict(m=-1.0), dict(m=nan), dict(to=(4096, 0)), dict(to=(4096, (1 << 20) + 1)), dict(to_types=(0, 5)),
                dict(to_types=(2, 1)), dict(ptrs=(4096, 4096)), dict(ptrs=(4096, 4112), types=(0, 0), to=(4096, 4112), to_types=(0, 0)),
                dict(to=(8192, 8208), to_types=(0, 1)), dict(to=(8192, 4104)), dict(to=(1 << 20, 4096))):
        assert clip(**bad) == fckl.ERR_ARG, bad
    assert clip(n=255) == fckl.ERR_WORKSPACE
    assert lib.fckl_clip_gradients(z, z, z, 1, 1.0, z, z, p, p, size(1), z) == fckl.ERR_ARG
    assert lib.fckl_launch_count() == before


def test_overlaps_that_are_refused(fckl):
    """Only what is written may overlap nothing: gradients that are read alone may lie in each other, in any
    order. (The workspace's size is checked after the lists, so that a list that passes gets that far.)"""
    lib = fckl.load()
    p, z, before = ctypes.c_void_p(4096), ctypes.c_void_p(0), lib.fckl_launch_count()

    def clip(ptrs, to, sizes):
        types = [fckl.F32] * len(ptrs)
        a, b, c, k = _arrays(ptrs, sizes, types)
        d, _, e, _ = _arrays(to, sizes, types)
        return lib.fckl_clip_gradients(a, b, c, k, 1.0, d, e, p, p, 0, z)

    A, B, C, D = 1 << 20, 1 << 21, 1 << 22, 1 << 23
    for ptrs, to, sizes in (((A, A), (C, D), (100, 100)), ((A, A + 40), (C, D), (100, 10)), ((A + 40, A), (D, C), (10, 100)),
                            ((A, B, A, A + 396), (C, B, D, C + 400), (100, 100, 100, 50)), ((A, A, A), (C, C + 400, D), (100, 100, 1)),
                            ((A,), (A,), (100,)), ((A, A), (A, C), (0, 100)), ((A, A, A + 20), (D, C, B), (100, 0, 10))):
        assert clip(ptrs, to, sizes) == fckl.ERR_WORKSPACE, (ptrs, to, sizes)
    for ptrs, to, sizes in (((A, A), (A, C), (100, 100)), ((A, A), (C, A), (100, 100)), ((A, A), (A, A), (100, 100)),
                            ((A, B), (C, C), (100, 100)), ((A, B), (C, C + 396), (100, 100)), ((A, B), (C + 396, C), (100, 100)),
                            ((A, A), (C, A + 396), (100, 100)), ((A, A + 4, B), (C, D, A + 200), (100, 10, 100)),
                            ((A, A + 40), (C, A + 40), (100, 10)), ((A, B), (C, C + 200), (100, 10)),
                            ((A, A + 8, A + 200), (C, D, A + 200), (100, 10, 1))):
        assert clip(ptrs, to, sizes) == fckl.ERR_ARG, (ptrs, to, sizes)
    assert lib.fckl_launch_count() == before


@gpu
def test_a_gradient_listed_twice(fckl):
    """Into other tensors: it counts twice, as in gradient_norm. A view of it as well."""
    a, b = tensor((300, 7), "fp32", 1), tensor((41,), "bf16", 2)
    grads = [a, b, a, a[10:20]]
    out = [torch.empty(g.shape, dtype=g.dtype, device="cuda") for g in grads]
    norm = fckl.clip_gradients(grads, 1.0, out=out)
    check_norm(norm, grads)
    check_scaled(out, grads, 1.0)
    assert torch.equal(norm, fckl.gradient_norm(grads)) and torch.equal(out[0], out[2])


@pytest.mark.parametrize("bad", [
    lambda f, g: f.gradient_norm([g]), lambda f, g: f.clip_gradients([g], 1.0), lambda f, g: f.clip_gradients([g], -1.0),
    lambda f, g: f.clip_gradients([g], float("nan")), lambda f, g: f.clip_gradients([g], 1.0, out=[]),
    lambda f, g: f.clip_gradients([g, None], 1.0, out=[g, g]),
])
def test_binding_refusals(fckl, bad, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises((TypeError, ValueError)):
        bad(fckl, torch.zeros(6, 8))


def test_lists_that_the_library_reads(fckl):
    """Types, layouts and devices of the tensors, without a GPU."""
    from chunked_kl_loss_gb300 import gradient_clip as m
    cpu = torch.device("cpu")
    a, b = torch.zeros(4, 6), torch.zeros(5, dtype=torch.bfloat16)
    some = [a, b, a.t(), a[1:3]]
    (ptrs, types, contiguous), sizes = m._list("grads", some, cpu), m._sizes(some)
    assert not contiguous and m._list("grads", [a, b], cpu)[2]
    assert list(ptrs) == [a.data_ptr(), b.data_ptr(), a.data_ptr(), a[1:].data_ptr()]
    assert list(sizes) == [24, 5, 24, 12] and list(types) == [fckl.F32, fckl.BF16, fckl.F32, fckl.F32]
    for bad in (a[:, 1:], a[::2], a[:, :1].expand(4, 3), torch.zeros(3).expand(2, 3)):
        with pytest.raises(ValueError):
            m._list("grads", [bad], cpu)
    for bad in (a.double(), a.int()):
        with pytest.raises(TypeError):
            m._list("grads", [bad], cpu)
    with pytest.raises(ValueError):
        m._list("grads", [a], torch.device("meta"))


@gpu
def test_binding_refusals_on_the_gpu(fckl):
    g = torch.ones(6, 8, device="cuda")
    for bad in (lambda: fckl.clip_gradients([g, g], 1.0), lambda: fckl.clip_gradients([g, g[2:]], 1.0),
                lambda: fckl.clip_gradients([g], 1.0, out=[g.view(-1)]), lambda: fckl.clip_gradients([g[:3]], 1.0, out=[g[1:4]]),
                lambda: fckl.clip_gradients([g], 1.0, out=[torch.empty(8, 6, device="cuda").t()]),
                lambda: fckl.gradient_norm([g[:, 1:]]), lambda: fckl.gradient_norm([g.double()]),
                lambda: fckl.gradient_norm([g, g.cpu()])):
        with pytest.raises((TypeError, ValueError, fckl.FcklError)):
            bad()
    assert (g == 1).all()


# ------------------------------------------------------------------ the oracle (CPU)
def test_oracle_closed_forms():
    assert orc.norm([np.array([3.0]), np.array([[4.0]])]) == 5.0 and orc.norm([]) == 0.0
    n, c, out = orc.clip([np.array([3.0]), np.array([4.0])], 1.0)
    assert n == 5.0 and abs(c - 0.2) < 1e-6 and abs(orc.norm(out) - 1.0) < 1e-6
    assert orc.clip([np.array([3.0])], 4.0)[1] == 1.0
