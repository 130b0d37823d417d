"""What the norm of queries and keys promises beside its values: overlaps,
positions outside the tables, the reach of non-finite values."""
import ctypes

import pytest
import torch

import fft_long_convolution_gb300 as F
from _mixers import qk_norm, rel

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
B, T, D, WIDE = 2, 4, 64, 8  # views below are heads of one [B, T, WIDE, D] buffer
BUF, OTHER, GRAD = 1 << 20, 1 << 24, 1 << 28  # addresses that nothing reads: every call here is refused


def view(base, head):
    return F.View(base + head * D * 2, T * WIDE * D, WIDE * D, D)


def args(q, k, Hq, Hk):
    a = F.QKNormArgs()
    a.dtype, a.norm, a.D, a.R, a.interleaved, a.eps = 1, 0, D, 0, 0, 1e-6
    a.B, a.T, a.Hq, a.Hk, a.q, a.k = B, T, Hq, Hk, q, k
    return a


@pytest.mark.parametrize("hq,hk", [((0, 4), (2, 4)), ((0, 2), (0, 2)), ((3, 2), (0, 4)), ((0, 8), (7, 1)), ((5, 1), (0, 8))])
def test_shared_heads_in_place_are_refused(hq, hk):
    """Queries and keys in place (forward on themselves, backward on their
    gradients) while they have heads in common."""
    L = F.lib()
    q, k = view(BUF, hq[0]), view(BUF, hk[0])
    a = args(q, k, hq[1], hk[1])
    assert L.fftconv_qknorm_forward(ctypes.byref(a), q, k, None) == 1
    b = args(view(OTHER, 0), view(2 * OTHER, 0), hq[1], hk[1])
    assert L.fftconv_qknorm_backward(ctypes.byref(b), q, k, q, k, None, None, None, 0, None) == 1


@pytest.mark.parametrize("hq,hk", [((0, 4), (2, 4)), ((0, 2), (0, 2)), ((0, 8), (7, 1))])
def test_outputs_over_each_other_are_refused(hq, hk):
    L = F.lib()
    yq, yk = view(GRAD, hq[0]), view(GRAD, hk[0])
    a = args(view(BUF, 0), view(OTHER, 0), hq[1], hk[1])
    assert L.fftconv_qknorm_forward(ctypes.byref(a), yq, yk, None) == 1
    assert L.fftconv_qknorm_backward(ctypes.byref(a), view(2 * OTHER, 0), view(4 * OTHER, 0), yq, yk, None, None, None, 0,
                                     None) == 1


def test_one_output_in_place_over_the_other_input_is_refused():
    L = F.lib()
    a = args(view(BUF, 0), view(BUF, 2), 4, 4)
    assert L.fftconv_qknorm_forward(ctypes.byref(a), a.q, view(OTHER, 0), None) == 1


@pytest.mark.parametrize("dwq,dwk,scratch", [
    (BUF, None, 4 * GRAD), (None, OTHER, 4 * GRAD), (2 * GRAD, None, 4 * GRAD), (5 * GRAD, 5 * GRAD, 4 * GRAD),
    (5 * GRAD, 5 * GRAD + 128, 4 * GRAD), (4 * GRAD, None, 4 * GRAD), (5 * GRAD, None, BUF), (5 * GRAD, None, 3 * GRAD),
    (6 * GRAD, None, 4 * GRAD), (GRAD, None, 4 * GRAD)])
def test_weight_gradients_and_scratch_over_other_buffers_are_refused(dwq, dwk, scratch):
    """Over an input (BUF, OTHER), a given gradient (GRAD), an output (2 and 3
    GRAD), a weight (6 GRAD), each other."""
    L = F.lib()
    a = args(view(BUF, 0), view(OTHER, 0), 4, 4)
    a.wq = 6 * GRAD
    n = L.fftconv_qknorm_scratch_bytes(ctypes.byref(a))
    st = L.fftconv_qknorm_backward(ctypes.byref(a), view(GRAD, 0), view(GRAD, 4), view(2 * GRAD, 0), view(3 * GRAD, 0), dwq, dwk,
                                   scratch, n, None)
    assert st == 1


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["token-major", "head-major", "batch-inside"])
def test_slices_of_one_buffer(layout):
    """Disjoint heads of one buffer, in whatever order it is stored: both in
    place, one of them, and written to other slices of it."""
    dt, Hq, Hk = torch.bfloat16, 3, 2
    order = {"token-major": (0, 1, 2, 3), "head-major": (0, 2, 1, 3), "batch-inside": (1, 0, 2, 3)}[layout]
    back = [order.index(i) for i in range(4)]
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(B, T, 2 * (Hq + Hk), D, generator=gen).to(dt)
    plan = F.QKNorm(D, dt)
    ref = qk_norm(x, None, "rms", 1e-6)

    def fresh():
        y = x.permute(order).contiguous().cuda().permute(back)
        return y, y[:, :, :Hq], y[:, :, Hq:Hq + Hk], y[:, :, Hq + Hk:2 * Hq + Hk], y[:, :, 2 * Hq + Hk:]

    for way in range(4):
        y, q, k, sq, sk = fresh()
        to = [(q, k), (q, None), (None, k), (sq, sk)][way]
        qo, ko = plan.forward(q, k, qo=to[0], ko=to[1])
        assert rel(qo, ref[:, :, :Hq]) < U[dt] and rel(ko, ref[:, :, Hq:Hq + Hk]) < U[dt]
        untouched = {0: slice(Hq + Hk, None), 1: slice(Hq, None), 2: slice(Hq + Hk, None), 3: slice(0, Hq + Hk)}[way]
        assert torch.equal(y[:, :, untouched].cpu(), x[:, :, untouched])


@pytest.mark.parametrize("dwq,dwk", [(5 * GRAD + 2, None), (None, 5 * GRAD + 1)])
def test_weight_gradients_off_their_alignment_are_refused(dwq, dwk):
    L = F.lib()
    a = args(view(BUF, 0), view(OTHER, 0), 4, 4)
    n = L.fftconv_qknorm_scratch_bytes(ctypes.byref(a))
    for T_ in (T, 0):
        a.T = T_
        assert L.fftconv_qknorm_backward(ctypes.byref(a), view(GRAD, 0), view(GRAD, 4), view(2 * GRAD, 0), view(3 * GRAD, 0), dwq,
                                         dwk, 4 * GRAD, n, None) == 3


def tables(rows, R):
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(R // 2, dtype=torch.float64) / max(R // 2, 1))
    return ang.cos().float().cuda(), ang.sin().float().cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_positions_outside_the_tables_reach_every_gradient(inter):
    """A token without a table row has NaN outputs and gradients; the weights'
    gradients are sums over all tokens, so it reaches them too.  Other tokens
    keep their values."""
    dt, b, t, Hq, Hk, d, R = torch.bfloat16, 1, 4, 2, 1, 64, 32
    gen = torch.Generator().manual_seed(3)
    q, k, dq, dk = (torch.randn(b, t, h, d, generator=gen).to(dt).cuda() for h in (Hq, Hk, Hq, Hk))
    wq, wk = torch.ones(d).cuda(), torch.ones(d).cuda()
    cos, sin = tables(10, R)
    plan = F.QKNorm(d, dt, rotary=R, interleaved=inter)

    def both(pos):
        kw = dict(wq=wq, wk=wk, cos=cos, sin=sin, positions=torch.tensor([pos], dtype=torch.int32).cuda())
        return plan.forward(q, k, **kw) + plan.backward(dq, dk, q, k, **kw)

    good, bad = both([0, 3, 4, 9]), both([0, -1, 10, 9])
    for x, y in zip(good[:4], bad[:4]):
        assert bool(torch.isfinite(x).all()) and bool(torch.isnan(y[:, 1:3]).all())
        assert torch.equal(x[:, [0, 3]], y[:, [0, 3]])
    for x, y in zip(good[4:], bad[4:]):
        assert bool(torch.isfinite(x).all()) and bool(torch.isnan(y).all())


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["weight", "input", "gradient"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("d,R,inter", [(64, 32, False), (64, 32, True), (24, 6, True), (24, 6, False), (96, 40, False), (80, 4, True)])
def test_unrotated_features_stay_by_themselves(d, R, inter, bad, what):
    """A NaN or an infinity in a feature past the rotated ones is mixed with no
    other feature: in a weight it is seen in that feature's output alone, in an
    input as the norm carries it, in a gradient in that weight's gradient alone."""
    dt, b, t, H, f = torch.bfloat16, 1, 3, 2, R
    gen = torch.Generator().manual_seed(4)
    q, k, dq, dk = (torch.randn(b, t, H, d, generator=gen).to(dt).cuda() for _ in range(4))
    wq, wk = torch.ones(d).cuda(), torch.ones(d).cuda()
    cos, sin = tables(10, R)
    plan = F.QKNorm(d, dt, rotary=R, interleaved=inter)
    kw = dict(cos=cos, sin=sin)
    others = [i for i in range(d) if i != f]
    if what == "weight":
        want, _ = plan.forward(q, k, wq=wq, wk=wk, **kw)
        wq[f] = bad
        got, _ = plan.forward(q, k, wq=wq, wk=wk, **kw)
        assert not bool(torch.isfinite(got[..., f]).any()) and torch.equal(got[..., others], want[..., others])
    elif what == "input":
        q[0, 1, 0, f] = bad
        got, _ = plan.forward(q, k, wq=wq, wk=wk, **kw)
        pos = torch.arange(t)[None].expand(b, t)
        ref = qk_norm(q.cpu(), wq.cpu(), "rms", 1e-6, cos.cpu(), sin.cpu(), pos, inter)
        assert torch.equal(torch.isnan(got).cpu(), torch.isnan(ref))
    else:
        want = plan.backward(dq, dk, q, k, wq=wq, wk=wk, **kw)[2]
        dq[0, 1, 0, f] = bad
        got = plan.backward(dq, dk, q, k, wq=wq, wk=wk, **kw)[2]
        assert not bool(torch.isfinite(got[f])) and torch.equal(got[others], want[others])
