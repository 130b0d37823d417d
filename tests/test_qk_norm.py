"""Norm and rotation of queries and keys on the GPU against 64 bits.

Arithmetic is float32 with one rounding to 16 bits at the end, so outputs and
input gradients are within one rounding (u = 2^-8 for bf16, 2^-11 for fp16 at
most; root mean square about 0.43 u) and weight gradients, sums of n terms of mixed
sign in float32, within sqrt(n) 2^-24 of a few times their terms: 2e-5.
"""
import ctypes

import pytest
import torch

import fft_long_convolution_gb300 as F
from _mixers import qk_norm, rel

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
DTYPES = [torch.bfloat16, torch.float16]


def tables(rows, R, seed=0):
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(R // 2, dtype=torch.float64) / max(R // 2, 1))
    return ang.cos().float().contiguous(), ang.sin().float().contiguous()


def inputs(B, T, Hq, Hk, D, dt, seed=0):
    gen = torch.Generator().manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=gen)
    return [mk(B, T, Hq, D).to(dt), mk(B, T, Hk, D).to(dt), 1 + 0.2 * mk(D), 1 + 0.2 * mk(D), mk(B, T, Hq, D).to(dt),
            mk(B, T, Hk, D).to(dt), torch.randint(0, 40, (B, T), generator=gen).to(torch.int32)]


CASES = [(1, 1, 1, 1, 64, 64), (2, 5, 4, 2, 128, 128), (3, 7, 3, 1, 128, 32), (1, 33, 2, 2, 80, 40), (2, 3, 5, 5, 96, 0),
         (1, 4, 1, 3, 256, 256), (1, 9, 2, 0, 8, 8), (2, 2, 1, 1, 24, 6), (1, 700, 7, 5, 64, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("norm,inter", [("rms", False), ("l2", True), ("l2", False), ("rms", True)])
@pytest.mark.parametrize("B,T,Hq,Hk,D,R", CASES)
def test_forward_and_backward(B, T, Hq, Hk, D, R, norm, inter, dt):
    q, k, wq, wk, dq, dk, pos = inputs(B, T, Hq, Hk, D, dt, seed=D + T)
    cos, sin = tables(40, R)
    plan = F.QKNorm(D, dt, norm=norm, rotary=R, interleaved=inter)
    kw = {n: x.cuda() for n, x in dict(wq=wq, wk=wk, cos=cos, sin=sin, positions=pos).items()}
    qo, ko = plan.forward(q.cuda(), k.cuda(), **kw)
    got = plan.backward(dq.cuda(), dk.cuda(), q.cuda(), k.cuda(), **kw)
    for x, w, d, y, gx, gw in ((q, wq, dq, qo, got[0], got[2]), (k, wk, dk, ko, got[1], got[3])):
        x, w = x.double().requires_grad_(), w.double().requires_grad_()
        ref = qk_norm(x, w, norm, 1e-6, cos, sin, pos, inter)
        assert rel(y, ref.detach()) < U[dt]
        if x.numel() == 0:
            assert not bool(gw.any())
            continue
        rx, rw = torch.autograd.grad((ref * d.double()).sum(), [x, w])
        assert rel(gx, rx) < U[dt] and rel(gw, rw) < 2e-5


@pytest.mark.gpu
def test_gradient_against_differences():
    """Along the gradient, the slope of the 64-bit function by central
    differences (step 1e-4) is the gradient's norm."""
    dt, B, T, H, D, R = torch.float16, 1, 3, 2, 64, 64
    q, k, wq, wk, dq, dk, pos = inputs(B, T, H, H, D, dt, seed=1)
    cos, sin = tables(40, R)
    plan = F.QKNorm(D, dt, rotary=R)
    kw = {n: x.cuda() for n, x in dict(wq=wq, wk=wk, cos=cos, sin=sin, positions=pos).items()}
    gq, _, gw, _ = plan.backward(dq.cuda(), dk.cuda(), q.cuda(), k.cuda(), **kw)

    def loss(x, w):
        return float((qk_norm(x, w, "rms", 1e-6, cos, sin, pos) * dq.double()).sum())

    gq, gw = gq.double().cpu(), gw.double().cpu()
    h = 1e-4
    a, b = gq / gq.norm(), gw / gw.norm()
    x, w = q.double(), wq.double()
    assert abs((loss(x + h * a, w) - loss(x - h * a, w)) / (2 * h) - float(gq.norm())) < U[dt] * float(gq.norm())
    assert abs((loss(x, w + h * b) - loss(x, w - h * b)) / (2 * h) - float(gw.norm())) < 2e-5 * float(gw.norm())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
def test_zero_rows_missing_weights_and_default_positions(dt):
    B, T, H, D, R = 2, 6, 2, 64, 64
    q, k, *_ = inputs(B, T, H, H, D, dt, seed=2)
    q[0, 1] = 0.0
    cos, sin = tables(T, R)
    pos = torch.arange(T)[None].expand(B, T)
    for norm in ("rms", "l2"):
        plan = F.QKNorm(D, dt, norm=norm, rotary=R)
        qo, ko = plan.forward(q.cuda(), k.cuda(), cos=cos.cuda(), sin=sin.cuda())
        assert rel(qo, qk_norm(q, None, norm, 1e-6, cos, sin, pos)) < U[dt]
        assert rel(ko, qk_norm(k, None, norm, 1e-6, cos, sin, pos)) < U[dt]
        assert not bool(qo[0, 1].any())
        g = plan.backward(qo, ko, q.cuda(), k.cuda(), cos=cos.cuda(), sin=sin.cuda())
        assert g[2] is None and g[3] is None and bool(torch.isfinite(g[1]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("norm,inter", [("rms", False), ("l2", True)])
def test_weights_and_tables_off_16_bytes(norm, inter):
    """float32 weights and tables need their own alignment only."""
    dt, B, T, H, D, R = torch.bfloat16, 2, 9, 3, 64, 32
    q, k, wq, wk, dq, dk, pos = [x.cuda() for x in inputs(B, T, H, H, D, dt, seed=5)]
    cos, sin = (x.cuda() for x in tables(40, R))
    plan = F.QKNorm(D, dt, norm=norm, rotary=R, interleaved=inter)

    def shifted(x):
        return torch.cat([x.new_zeros(1), x.flatten()])[1:].view(x.shape)

    sets = [dict(wq=wq, wk=wk, cos=cos, sin=sin, positions=pos)]
    sets.append({n: x if n == "positions" else shifted(x) for n, x in sets[0].items()})
    res = [list(plan.forward(q, k, **kw)) + list(plan.backward(dq, dk, q, k, **kw)) for kw in sets]
    assert all(torch.equal(x, y) for x, y in zip(*res))


@pytest.mark.gpu
def test_positions_outside_the_tables_give_nan():
    dt, B, T, H, D, R = torch.bfloat16, 1, 4, 2, 64, 32
    q, k, *_ = inputs(B, T, H, H, D, dt, seed=3)
    cos, sin = tables(10, R)
    pos = torch.tensor([[0, -1, 10, 9]], dtype=torch.int32)
    plan = F.QKNorm(D, dt, rotary=R)
    qo, _ = plan.forward(q.cuda(), k.cuda(), cos=cos.cuda(), sin=sin.cuda(), positions=pos.cuda())
    assert bool(torch.isnan(qo[:, 1:3]).all()) and bool(torch.isfinite(qo[:, [0, 3]]).all())


@pytest.mark.gpu
def test_strides_in_place_and_streams():
    """Slices of one projection, in place and not, on a side stream."""
    dt, B, T, Hq, Hk, D, R = torch.bfloat16, 2, 50, 4, 2, 128, 64
    q, k, wq, wk, dq, dk, pos = [x.cuda() for x in inputs(B, T, Hq, Hk, D, dt, seed=4)]
    cos, sin = (x.cuda() for x in tables(40, R))
    kw = dict(wq=wq, wk=wk, cos=cos, sin=sin, positions=pos)
    plan = F.QKNorm(D, dt, rotary=R)
    want = plan.forward(q, k, **kw)
    wantg = plan.backward(dq, dk, q, k, **kw)
    both = torch.cat([q, k], 2)
    sq, sk = both[:, :, :Hq], both[:, :, Hq:]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = plan.forward(sq, sk, stream=side, **kw)
    gotg = plan.backward(dq, dk, sq, sk, stream=side, **kw)
    plan.forward(sq, sk, qo=sq, ko=sk, stream=side, **kw)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert all(torch.equal(x, y) for x, y in zip(wantg, gotg))
    assert torch.equal(want[0], sq) and torch.equal(want[1], sk)


def args(**kw):
    a = F.QKNormArgs()
    v = F.View(1 << 20, 4096, 1024, 64)
    a.dtype, a.norm, a.D, a.R, a.interleaved, a.eps = 1, 0, 64, 0, 0, 1e-6
    a.B, a.T, a.Hq, a.Hk = 2, 4, 2, 2
    a.q, a.k = v, F.View(1 << 24, 4096, 1024, 64)
    for n, x in kw.items():
        setattr(a, n, x)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(D=60), 2), (dict(D=264), 2), (dict(D=0), 2), (dict(R=7), 2), (dict(R=66), 2), (dict(R=-2), 2), (dict(dtype=3), 2),
    (dict(norm=2), 2), (dict(B=-1), 1), (dict(eps=float("nan")), 1), (dict(eps=-1.0), 1), (dict(R=64), 1),
    (dict(wq=2), 3), (dict(Hq=70000), 2), (dict(q=F.View((1 << 20) + 8, 4096, 1024, 64)), 3),
    (dict(q=F.View(1 << 20, 4096, 1020, 64)), 3), (dict(q=F.View(1 << 20, 0, 1024, 64)), 1), (dict(q=F.View(0, 4096, 1024, 64)), 1)])
def test_refusals_without_gpu(kw, status):
    L = F.lib()
    y1, y2 = F.View(1 << 26, 4096, 1024, 64), F.View(1 << 27, 4096, 1024, 64)
    assert L.fftconv_qknorm_forward(ctypes.byref(args(**kw)), y1, y2, None) == status


def test_overlaps_and_missing_scratch_without_gpu():
    L = F.lib()
    y1, y2 = F.View(1 << 26, 4096, 1024, 64), F.View(1 << 27, 4096, 1024, 64)
    a = args()
    assert L.fftconv_qknorm_forward(None, y1, y2, None) == 1
    # a shifted output over the input; the outputs exchanged
    assert L.fftconv_qknorm_forward(ctypes.byref(a), F.View((1 << 20) + 64, 4096, 1024, 64), y2, None) == 1
    assert L.fftconv_qknorm_forward(ctypes.byref(a), a.k, a.q, None) == 1
    d1, d2 = F.View(1 << 28, 4096, 1024, 64), F.View(1 << 29, 4096, 1024, 64)
    assert L.fftconv_qknorm_backward(ctypes.byref(a), d1, d2, y1, y2, 1 << 30, None, None, 0, None) == 4
    n = L.fftconv_qknorm_scratch_bytes(ctypes.byref(a))
    assert n > 0 and L.fftconv_qknorm_scratch_bytes(ctypes.byref(args(D=60))) == 0
    # nothing to do
    assert L.fftconv_qknorm_forward(ctypes.byref(args(T=0)), y1, y2, None) == 0


def test_binding_refusals_without_gpu():
    with pytest.raises(ValueError):
        F.QKNorm(64, torch.bfloat16, norm="layer")
    with pytest.raises(TypeError):
        F.QKNorm(64, torch.float32)
    x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        F.QKNorm(64, torch.bfloat16).forward(x, x)
