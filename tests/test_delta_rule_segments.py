"""Rows that are cut into segments: with a backward behind them, packed, with
shared key heads, at every head size.  Tolerances as in the tests of short rows
(u = 2^-8 for bf16, 2^-11 for fp16): states 2e-5, outputs 1.25 u, gradients
1.5 u, of the gates 3 u.  The 64-bit side runs on the GPU."""
import pytest
import torch

import fft_long_convolution_gb300 as F
from _mixers import delta_inputs, rel

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
DTYPES = [torch.bfloat16, torch.float16]
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dstate")


def rule(q, k, v, g, beta, S, scale):
    """The definition in float64, token by token (tests/_mixers.py, on the tensors' device)."""
    group = g.shape[2] // q.shape[2]
    q, k = (x.repeat_interleave(group, 2) for x in (q, k))
    a, outs = g.exp()[..., None, None], []
    for t in range(q.shape[1]):
        S = S * a[:, t]
        u = beta[:, t, :, None] * (v[:, t] - (k[:, t, :, None] @ S)[:, :, 0])
        S = S + k[:, t, :, :, None] * u[:, :, None]
        outs.append((q[:, t, :, None] @ S)[:, :, 0])
    return scale * torch.stack(outs, 1), S


def expected(ins, do, s0, ds, scale):
    """Outputs, final states and gradients of one batch of equal rows."""
    xs = [x.cuda().double().requires_grad_() for x in (*ins, s0)]
    o, s = rule(*xs, scale)
    grads = torch.autograd.grad((o * do.cuda().double()).sum() + (s * ds.cuda().double()).sum(), xs)
    return [x.detach().cpu() for x in (o, s, *grads)]


def states(n, H, Dk, Dv, seed):
    return 0.3 * torch.randn(n, H, Dk, Dv, generator=torch.Generator().manual_seed(seed))


def cut(plan, B, T, Hk, Hv, nseq):
    """Whether these rows are cut: only then a forward that saves needs scratch."""
    return F.lib().fftconv_delta_scratch_bytes(plan._h, B, T, Hk, Hv, nseq, 2) > 0


def tol(name, dt):
    return (3 if name in ("dg", "dbeta") else 1.5) * U[dt]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("B,T,Hk,Hv,Dk,Dv", [(1, 4000, 1, 3, 128, 128), (2, 4100, 1, 1, 64, 64), (1, 4097, 2, 2, 64, 128),
                                             (1, 3968, 1, 2, 128, 64)])
def test_rows(B, T, Hk, Hv, Dk, Dv, dt):
    ins = delta_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=T)
    do = delta_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=T + 1)[2]
    s0, ds = states(B, Hv, Dk, Dv, 1), states(B, Hv, Dk, Dv, 2)
    plan = F.DeltaRule(Dk, Dv, dt)
    assert cut(plan, B, T, Hk, Hv, B)
    dins = [x.cuda() for x in ins]
    o, s, saved = plan.forward(*dins, state=s0.cuda(), save=True)
    got = plan.backward(do.cuda(), *dins, saved, dstate=ds.cuda())
    assert plan.device_status() == 0
    ref = expected(ins, do, s0, ds, Dk ** -0.5)
    assert rel(o, ref[0]) < 1.25 * U[dt] and rel(s, ref[1]) < 2e-5
    for name, x, y in zip(NAMES, got, ref[2:]):
        assert rel(x, y) < tol(name, dt), name
    plain, s2 = plan.forward(*dins, state=s0.cuda())
    assert torch.equal(plain, o) and torch.equal(s2, s)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("Hk,Hv,Dk,Dv", [(1, 1, 128, 128), (1, 2, 64, 128)])
def test_packed(Hk, Hv, Dk, Dv, dt):
    """Sequences of several segments, an empty one, one shorter than a segment;
    tokens after the last belong to none."""
    lens = [7000, 0, 100, 6000]
    T, n = sum(lens) + 3, len(lens)
    ins = delta_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=5)
    do = delta_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=6)[2]
    s0, ds = states(n, Hv, Dk, Dv, 3), states(n, Hv, Dk, Dv, 4)
    off = torch.zeros(n + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(torch.tensor(lens), 0)
    plan = F.DeltaRule(Dk, Dv, dt)
    assert cut(plan, 1, T, Hk, Hv, n)
    dins = [x.cuda() for x in ins]
    o, s, saved = plan.forward(*dins, state=s0.cuda(), offsets=off.cuda(), save=True)
    got = plan.backward(do.cuda(), *dins, saved, dstate=ds.cuda(), offsets=off.cuda())
    assert plan.device_status() == 0
    for i, L in enumerate(lens):
        at = slice(int(off[i]), int(off[i]) + L)
        if L == 0:
            assert torch.equal(s[i].cpu(), s0[i]) and torch.equal(got[5][i].cpu(), ds[i])
            continue
        ref = expected([x[:, at] for x in ins], do[:, at], s0[i:i + 1], ds[i:i + 1], Dk ** -0.5)
        assert rel(o[:, at], ref[0]) < 1.25 * U[dt] and rel(s[i:i + 1], ref[1]) < 2e-5
        for name, x, y in zip(NAMES[:5], got, ref[2:]):
            assert rel(x[:, at], y) < tol(name, dt), (name, i)
        assert rel(got[5][i:i + 1], ref[7]) < tol("dstate", dt)
    assert all(not bool(x[:, sum(lens):].any()) for x in (o, *got[:5]))
