"""Gated delta rule where its intermediate sums are far larger than its results.

The tolerances are those of the ordinary inputs (u = 2^-8 for bf16, 2^-11 for
fp16): states 2e-5, outputs 1.25 u, gradients 1.5 u, of the gates 3 u; heads are
compared one by one where their decays matter.
"""
import pytest
import torch

import fft_long_convolution_gb300 as F
from _mixers import delta_inputs, delta_rule, rel

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
DTYPES = [torch.bfloat16, torch.float16]
NAMES = ("dq", "dk", "dv", "dg", "dbeta")


def gradients(ins, do, scale):
    xs = [x.double().requires_grad_() for x in ins]
    o, _ = delta_rule(*xs, scale=scale)
    return torch.autograd.grad((o * do.double()).sum(), xs)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("low", [float("-inf"), -60.0, -20.0])
@pytest.mark.parametrize("n", [16, 40])
def test_many_resets_in_one_chunk(n, low, dt):
    """n tokens in a row that empty the state (or nearly), then weak decays in
    the same chunk: the decays between the latter do not feel the former."""
    B, T, H, D = 1, 192, 3, 128
    q, k, v, g, beta = delta_inputs(B, T, H, H, D, D, dt, seed=n)
    g[:, 128:128 + n] = low
    ins = (q, k, v, g, beta)
    do = delta_inputs(B, T, H, H, D, D, dt, seed=n + 1)[2]
    plan = F.DeltaRule(D, D, dt)
    dins = [x.cuda() for x in ins]
    o, s, saved = plan.forward(*dins, save=True)
    got = plan.backward(do.cuda(), *dins, saved)
    fin = [x.double() for x in ins]
    fin[3] = fin[3].clamp(min=-200.0)
    ref, sref = delta_rule(*fin, scale=D ** -0.5)
    r = gradients(fin, do, D ** -0.5)
    for h in range(H):
        assert rel(s[:, h], sref[:, h]) < 2e-5
        assert rel(o[:, :, h], ref[:, :, h]) < 1.25 * U[dt]
        for name, x, y in zip(NAMES, got, r):
            assert rel(x[:, :, h], y[:, :, h]) < (3 if name in ("dg", "dbeta") else 1.5) * U[dt], name


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
def test_gate_gradients_with_alike_keys(dt):
    """Keys with a cosine of 0.9 to one another and beta = 0.9, which is no power
    of two: what a pair of tokens adds to one end of dg's sum and takes from the
    other has to be the same number."""
    B, T, H, D = 2, 130, 4, 128
    q, k, v, g, beta = delta_inputs(B, T, H, H, D, D, dt, seed=61)
    gen = torch.Generator().manual_seed(62)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    k = n(B, T, H, D) + 3.0 * n(B, 1, H, D)
    q = n(B, T, H, D)
    q, k = ((x / x.norm(dim=-1, keepdim=True)).to(dt) for x in (q, k))
    beta = torch.full_like(beta, 0.9)
    ins = (q, k, v, g, beta)
    do = delta_inputs(B, T, H, H, D, D, dt, seed=63)[2]
    plan = F.DeltaRule(D, D, dt)
    dins = [x.cuda() for x in ins]
    _, _, saved = plan.forward(*dins, save=True)
    got = plan.backward(do.cuda(), *dins, saved)
    r = gradients(ins, do, D ** -0.5)
    assert rel(got[3], r[3]) < 3 * U[dt]
