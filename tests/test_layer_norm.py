"""Layer norm on the GPU against its 64-bit definition.

Tolerances (2-norm of the difference over that of the result).  y and dx: float32
and one rounding to 16 bits, at most u = 2^-8 (bf16) or 2^-11 (fp16) of an element.
dw, db: float32 sums of float32 terms; a term is good to 4 2^-24, a sum over n
tokens is taken in runs of at most n / (groups of lanes) and in trees above, so its
error is a few 2^-24 of the sum of the terms' sizes, sqrt(n) times the result for
terms of either sign, over sqrt(n) for errors of either sign: 2e-6 holds 30 2^-24.
"""
import ctypes

import pytest
import torch

import fft_long_convolution_gb300 as F
from _attention import layer_norm, rel

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
DTYPES = [torch.bfloat16, torch.float16]
TOL_W = 2e-6


def inputs(shape, dt, seed=0):
    gen = torch.Generator().manual_seed(seed)

    def n(*s):
        return torch.randn(*s, generator=gen, dtype=torch.float64)

    ws = shape[-1:] if len(shape) < 4 else shape[-2:]
    x = (n(*shape) * (0.5 + n(*ws).abs()) + n(*ws)).to(dt)
    return x, (1.0 + 0.3 * n(*ws)).float(), (0.2 * n(*ws)).float(), n(*shape).to(dt)


def grads(x, w, b, dy, eps=1e-5):
    xs = [t.double().requires_grad_() for t in (x, w, b)]
    return torch.autograd.grad((layer_norm(*xs, eps=eps) * dy.double()).sum(), xs)


# every way a row is held (lanes, runs), at its first and last size, odd row counts
SHAPES = [(1, 1, 8), (3, 33, 16), (2, 129, 32), (1, 5, 40), (2, 77, 64), (1, 9, 72), (1, 200, 128), (2, 17, 136), (1, 130, 256),
          (1, 35, 264), (3, 11, 512), (1, 7, 520), (2, 50, 768), (1, 3, 776), (1, 19, 1024), (1, 6, 1032), (2, 3, 2048),
          (1, 5, 2056), (1, 4, 4096), (1, 3, 4104), (1, 2, 5000), (1, 3, 6152), (2, 2, 8192), (2, 65, 3, 64), (3, 5, 12, 128),
          (1, 41, 5, 80), (1, 2, 7, 1032), (700, 40), (1, 768)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, dt):
    x, w, b, dy = inputs(shape, dt, seed=sum(shape))
    norm = F.LayerNorm(shape[-1], dt)
    y = norm.forward(x.cuda(), w.cuda(), b.cuda())
    assert y.dtype == dt and y.shape == x.shape
    assert rel(y, layer_norm(x, w, b)) < U[dt]
    got = norm.backward(dy.cuda(), x.cuda(), w.cuda(), b.cuda())
    for name, g, r, t in zip(("dx", "dw", "db"), got, grads(x, w, b, dy), (U[dt], TOL_W, TOL_W)):
        assert g.shape == r.shape and rel(g, r) < t, name
    again = norm.backward(dy.cuda(), x.cuda(), w.cuda(), b.cuda())
    assert all(torch.equal(p, q) for p, q in zip(got, again))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("D", [64, 768, 2048])
@pytest.mark.parametrize("which", ["", "w", "b"])
def test_missing_weights(D, which, dt):
    x, w, b, dy = inputs((2, 37, D), dt, seed=D)
    w, b = (w if "w" in which else None), (b if "b" in which else None)
    dev = [None if t is None else t.cuda() for t in (w, b)]
    norm = F.LayerNorm(D, dt)
    assert rel(norm.forward(x.cuda(), *dev), layer_norm(x, w, b)) < U[dt]
    dx, dw, db = norm.backward(dy.cuda(), x.cuda(), *dev)
    r = grads(x, torch.ones(D) if w is None else w, torch.zeros(D) if b is None else b, dy)
    assert rel(dx, r[0]) < U[dt]
    assert dw is None if w is None else rel(dw, r[1]) < TOL_W
    assert db is None if b is None else rel(db, r[2]) < TOL_W


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(6, 40000, 32), (3, 4001, 768), (2, 3000, 4, 64)])
def test_many_rows(shape):
    """More rows than the backward's CTAs take at once."""
    dt = torch.bfloat16
    x, w, b, dy = inputs(shape, dt, seed=5)
    norm = F.LayerNorm(shape[-1], dt)
    assert rel(norm.forward(x.cuda(), w.cuda(), b.cuda()), layer_norm(x, w, b)) < U[dt]
    for g, r, t in zip(norm.backward(dy.cuda(), x.cuda(), w.cuda(), b.cuda()), grads(x, w, b, dy), (U[dt], TOL_W, TOL_W)):
        assert rel(g, r) < t


@pytest.mark.gpu
def test_backward_against_differences():
    """Slopes of the 64-bit definition along the gradient, by central differences
    of step 1e-4 of the input's size (truncation 1e-8)."""
    dt, shape = torch.float16, (2, 5, 72)
    x, w, b, dy = inputs(shape, dt, seed=9)
    got = F.LayerNorm(72, dt).backward(dy.cuda(), x.cuda(), w.cuda(), b.cuda())
    xs = [t.double() for t in (x, w, b)]
    for i, g in enumerate(got):
        g = g.double().cpu()
        step = 1e-4 * float(xs[0].norm()) * g / g.norm()
        vals = [float((layer_norm(*[t + s * step if j == i else t for j, t in enumerate(xs)]) * dy.double()).sum()) for s in (1, -1)]
        slope = (vals[0] - vals[1]) / (2 * float(step.norm()))
        assert abs(slope - float(g.norm())) < U[dt] * float(g.norm()), i


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 768, 2048])
def test_large_means_and_flat_rows(D):
    """A mean of 200 spreads (the variance would lose all its digits as a difference
    of squares), a row of equal values (y is b), eps that outweighs the variance."""
    dt = torch.float16
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(1, 20, D, generator=gen) + 200.0
    x[:, 3] = 7.0
    x = x.to(dt)
    b = torch.randn(D, generator=gen)
    norm = F.LayerNorm(D, dt)
    y = norm.forward(x.cuda(), None, b.cuda())
    assert rel(y, layer_norm(x, None, b)) < U[dt]
    assert torch.equal(y[0, 3].cpu(), b.to(dt))
    big = F.LayerNorm(D, dt, eps=1e4)
    assert rel(big.forward(x.cuda()), layer_norm(x, eps=1e4)) < U[dt]


@pytest.mark.gpu
@pytest.mark.parametrize("D", [32, 768, 4096])
def test_non_finite_rows_stay_alone(D):
    dt = torch.bfloat16
    x, w, b, dy = (t.cuda() for t in inputs((1, 50, D), dt, seed=3))
    norm = F.LayerNorm(D, dt)
    y0, dx0 = norm.forward(x, w, b), norm.backward(dy, x, w, b)[0]
    bad = x.clone()
    bad[0, 7, 3], bad[0, 21, D - 1] = float("nan"), float("inf")
    y1, (dx1, dw, db) = norm.forward(bad, w, b), norm.backward(dy, bad, w, b)
    keep = [i for i in range(50) if i not in (7, 21)]
    assert torch.equal(y0[:, keep], y1[:, keep]) and torch.equal(dx0[:, keep], dx1[:, keep])
    for t in (y1, dx1):
        assert bool(t[0, [7, 21]].isnan().all())
    assert bool(dw.isnan().any()) and bool(db.isfinite().all())


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2, 33, 64), (2, 9, 768), (1, 5, 2048), (2, 21, 3, 64)])
def test_in_place_strides_and_streams(shape):
    """Outputs over the input, slices of a wider buffer, batch-minor storage, weights
    off a 16-byte boundary, a side stream: the bits of contiguous tensors."""
    dt, D = torch.bfloat16, shape[-1]
    x, w, b, dy = (t.cuda() for t in inputs(shape, dt, seed=4))
    norm = F.LayerNorm(D, dt)
    y, (dx, dw, db) = norm.forward(x, w, b), norm.backward(dy, x, w, b)
    z = x.clone()
    assert norm.forward(z, w, b, y=z) is z and torch.equal(z, y)
    wide = torch.full((*shape[:-1], 2 * D + 8), 7.0, dtype=dt, device="cuda")
    left, right = wide[..., :D], wide[..., D + 8:]
    left.copy_(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    norm.forward(left, w, b, y=right, stream=side)
    side.synchronize()
    assert torch.equal(right, y) and torch.equal(left, x) and bool((wide[..., D:D + 8] == 7.0).all())
    xt, dyt = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (x, dy))
    off = torch.zeros(w.numel() + 1, device="cuda")[1:].view(w.shape).copy_(w)
    g = norm.backward(dyt, xt, off, b)
    assert torch.equal(norm.forward(xt, off, b), y)
    assert all(torch.equal(p, q) for p, q in zip(g, (dx, dw, db)))


@pytest.mark.gpu
def test_empty_calls():
    norm = F.LayerNorm(64, torch.bfloat16)
    w = torch.ones(64, device="cuda")
    x = torch.empty(2, 0, 64, dtype=torch.bfloat16, device="cuda")
    assert norm.forward(x, w, w).shape == x.shape
    torch.full((64,), 3.0, device="cuda")
    dx, dw, db = norm.backward(x, x, w, w)
    assert dx.shape == x.shape and not bool(dw.any()) and not bool(db.any())
    x = torch.empty(2, 3, 0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(0, 64, device="cuda")
    assert norm.forward(x, w, w).numel() == 0 and norm.backward(x, x, w, w)[1].numel() == 0


@pytest.mark.gpu
def test_captured_calls_replay():
    dt, shape = torch.bfloat16, (3, 301, 768)
    norm = F.LayerNorm(768, dt)
    first, second = ([t.cuda() for t in inputs(shape, dt, seed=s)] for s in (6, 7))
    held = [t.clone() for t in first]

    def work(x, w, b, dy):
        return [norm.forward(x, w, b), *norm.backward(dy, x, w, b)]

    work(*held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = work(*held)
    for ins in (first, second):
        for p, q in zip(held, ins):
            p.copy_(q)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(kept, work(*ins)))


@pytest.mark.gpu
def test_refused_tensors():
    dt = torch.bfloat16
    norm = F.LayerNorm(64, dt)
    x = torch.zeros(2, 5, 64, dtype=dt, device="cuda")
    w = torch.ones(64, device="cuda")
    for bad in (lambda: norm.forward(x.float()), lambda: norm.forward(x[..., :32]), lambda: norm.forward(x, w[:32]),
                lambda: norm.forward(x, w.half()), lambda: norm.forward(x, w.cpu()), lambda: norm.forward(x.cpu()),
                lambda: norm.forward(x, y=x[:1]), lambda: norm.backward(x[:, :2], x), lambda: norm.forward(x[0, 0]),
                lambda: norm.forward(x.unsqueeze(2), w)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(F.FFTConvError) as e:
        norm.forward(torch.zeros(2, 5, 72, dtype=dt, device="cuda")[..., 4:68])
    assert e.value.status == 3
    with pytest.raises(F.FFTConvError) as e:
        norm.forward(x[:1].expand(2, -1, -1))
    assert e.value.status == 1


BUF, OTHER, GRAD = 1 << 20, 1 << 24, 1 << 28  # addresses that nothing reads: every call below is refused
B, T, H, D = 2, 4, 3, 64


def args(x=BUF, w=None, b=None, **kw):
    a = F.LayerNormArgs()
    a.dtype, a.D, a.eps, a.B, a.T, a.H = 1, D, 1e-5, B, T, H
    a.x, a.w, a.b = view(x), w, b
    for k, v in kw.items():
        setattr(a, k, v)
    return ctypes.byref(a)


def view(base):
    return F.View(base, T * H * D, H * D, D)


@pytest.mark.parametrize("want,kw", [(2, dict(D=0)), (2, dict(D=12)), (2, dict(D=8200)), (2, dict(dtype=3)), (1, dict(eps=-1.0)),
                                     (1, dict(eps=float("nan"))), (1, dict(B=-1)), (2, dict(H=65536)), (2, dict(T=1 << 30)),
                                     (2, dict(B=1 << 20, T=1 << 10)), (2, dict(B=1 << 10, T=1 << 10, H=1 << 10)), (3, dict(w=OTHER + 2)),
                                     (3, dict(x=F.View(BUF + 8, T * H * D, H * D, D))), (3, dict(x=F.View(BUF, T * H * D, H * D, D + 4))),
                                     (1, dict(x=F.View(BUF, T * H * D, 0, D))), (1, dict(x=F.View(None, 1, 1, 1)))])
def test_refused_arguments(want, kw):
    L = F.lib()
    a = F.LayerNormArgs()
    a.dtype, a.D, a.eps, a.B, a.T, a.H, a.x = 1, D, 1e-5, B, T, H, view(BUF)
    for k, v in kw.items():
        setattr(a, k, v)
    assert L.fftconv_layernorm_forward(ctypes.byref(a), view(GRAD), None) == want
    assert L.fftconv_layernorm_backward(ctypes.byref(a), view(2 * GRAD), view(GRAD), None, None, None, 0, None) == want
    assert L.fftconv_layernorm_forward(None, view(GRAD), None) == 1
    assert L.fftconv_layernorm_scratch_bytes(None) == 0


def test_overlaps_are_refused():
    L = F.lib()
    assert L.fftconv_layernorm_forward(args(), view(BUF + 16), None) == 1  # shifted by 8 features
    assert L.fftconv_layernorm_forward(args(w=OTHER), view(OTHER), None) == 1
    assert L.fftconv_layernorm_forward(args(b=OTHER), view(OTHER - 1024), None) == 1
    need = L.fftconv_layernorm_scratch_bytes(args())
    back = lambda dy, dx, dw, db, scratch, n=need, **kw: L.fftconv_layernorm_backward(  # noqa: E731
        args(**kw), view(dy), view(dx), dw, db, scratch, n, None)
    free = dict(dy=2 * GRAD, dx=GRAD, dw=3 * GRAD, db=4 * GRAD, scratch=5 * GRAD)
    assert back(**free, n=need - 1) == 4 and back(**{**free, "scratch": None}) == 4
    assert back(**{**free, "scratch": 5 * GRAD + 8}) == 3 and back(**{**free, "dw": 3 * GRAD + 2}) == 3
    assert back(**{**free, "dx": 2 * GRAD + 16}) == 1 and back(**{**free, "dx": BUF + 128}) == 1
    for name in ("dw", "db", "scratch"):
        for over in (BUF, GRAD, 2 * GRAD, OTHER):
            assert back(**{**free, name: over}, w=OTHER) == 1, (name, over)
    assert back(**{**free, "db": 3 * GRAD + 64}) == 1 and back(**{**free, "dw": 5 * GRAD}) == 1
    assert L.fftconv_layernorm_backward(args(T=0), view(GRAD), view(GRAD), OTHER, OTHER, None, 0, None) == 1
