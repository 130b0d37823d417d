"""How far outputs and states may be off, element by element, where the norms of the
other tests say little: outputs whose terms cancel, values at the bottom of fp16."""
import pytest
import torch

import fft_long_convolution_gb300 as F
from _attention import attention_inputs, linear_attention, states

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
C = 64  # tokens that share a copy of the state


def sizes(q, k, v, decay, state):
    """For rows of one head: the definition's (o, final state), and the sum of its terms'
    sizes as the copies of the state and the scores enter it, scale 1, in 64 bits."""
    q, k, v, S = (x.double() for x in (q, k, v, state))
    lam, T = float(decay.double().exp()), q.shape[0]
    o, size = torch.zeros(T, v.shape[1], dtype=torch.float64), torch.zeros(T, v.shape[1], dtype=torch.float64)
    for s in range(0, T, C):
        x, y, z = (a[s:s + C] for a in (q, k, v))
        i = torch.arange(x.shape[0], dtype=torch.float64)
        u = (lam ** (i + 1))[:, None]
        P = (x @ y.T) * torch.tril(lam ** (i[:, None] - i).clamp(min=0))
        o[s:s + C] = u * (x @ S) + P @ z
        size[s:s + C] = u * (x.abs() @ S.abs()) + P.abs() @ z.abs()
        S = lam ** len(i) * S + (y * (lam ** (len(i) - 1 - i))[:, None]).T @ z
    return o, S, size


def test_sizes_are_of_the_definition():
    ins = attention_inputs(1, 150, 1, 1, 64, 128, torch.bfloat16, seed=2)
    s0 = states(1, 1, 64, 128)
    ref, sref = linear_attention(*ins, s0)
    o, S, size = sizes(*(x[0, :, 0] for x in ins[:3]), ins[3], s0[0, 0])
    assert torch.allclose(o, ref[0, :, 0], rtol=1e-12, atol=1e-9) and torch.allclose(S, sref[0, 0], rtol=1e-12, atol=1e-9)
    assert bool((size >= o.abs()).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", U)
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128)])
@pytest.mark.parametrize("cancel", [False, True])
def test_outputs_within_their_terms(cancel, Dk, Dv, dt):
    """o is off by u (|o| + the sum of its terms' sizes): the last rounding, that of S and
    that of P, each at most u of what it rounds.  What feeds S (17 bits, 2^-17 of it) and
    float32's sums (at most 16 additions a chunk, 2^-23 each, 3 chunks) add less than u / 64
    of the same sizes in either type.  With cancel, tokens of the second chunk overwrite what
    the state holds under their keys, so that o is a small part of its terms."""
    T, scale = 3 * C - 5, Dk ** -0.5
    q, k, v, _ = attention_inputs(1, T, 1, 1, Dk, Dv, dt, seed=Dk)
    s0, decay = states(1, 1, Dk, Dv), torch.tensor([-2.0 ** -7])
    if cancel:
        S, lam = linear_attention(q[:, :C], k[:, :C], v[:, :C], decay, s0)[1][0, 0], float(decay.double().exp())
        for t in range(C, C + 20):
            q[0, t] = k[0, t]
            key = k[0, t, 0].double()
            v[0, t, 0] = (-lam * (S.T @ key) / (key @ key)).to(dt)
            S = lam * S + key[:, None] * v[0, t, 0].double()
    plan = F.LinearAttention(Dk, Dv, dt)
    o, _ = plan.forward(*(x.cuda() for x in (q, k, v)), decay.cuda(), state=s0.cuda())
    ref, _, size = sizes(*(x[0, :, 0] for x in (q, k, v)), decay, s0[0, 0])
    ref, size = scale * ref, scale * size
    got = o[0, :, 0].double().cpu()
    if cancel:
        few = slice(C, C + 20)
        assert float(ref[few].norm()) < float(size[few].norm()) / 100
    assert bool(((got - ref).abs() <= U[dt] * (ref.abs() + (1 + 2.0 ** -6) * size)).all())
    assert plan.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("exponent", [-24, -23, -21, -19, -17])
def test_fp16_states_of_values_at_the_bottom(exponent):
    """Values of at most 2^exponent (subnormal in fp16), scaled by at most 2^15 on their way
    into a state, where the roundings of their two parts are 2^-25 each: 2^-39 a token.  A
    weight is within 2^-25, the product's parts within 2^-21 of it; doubled for the sums."""
    dt, T, D = torch.float16, 150, 64
    q, k, v, decay = attention_inputs(1, T, 1, 1, D, D, dt, seed=31)
    gen = torch.Generator().manual_seed(exponent)
    top = 2 ** (exponent + 24)
    v = (torch.randint(-top, top + 1, v.shape, generator=gen).double() * 2.0 ** -24).to(dt)
    ref = linear_attention(q, k, v, decay)[1][0, 0]
    plan = F.LinearAttention(D, D, dt)
    s = plan.forward(q.cuda(), k.cuda(), v.cuda(), decay.cuda())[1].cpu().double()[0, 0]
    w = (decay.double() * (T - 1 - torch.arange(T, dtype=torch.float64))).exp()
    a, b = k[0, :, 0].double().abs(), v[0, :, 0].double().abs()
    off = torch.einsum("tk,tv,t->kv", a, b, 2.0 ** -25 + 2.0 ** -21 * w) + 2.0 ** -39 * a.sum(0)[:, None]
    assert bool(((s - ref).abs() <= 2 * off).all())
    assert plan.device_status() == 0
