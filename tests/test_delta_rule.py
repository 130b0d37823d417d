"""Gated delta rule on the GPU against its 64-bit definition.

Tolerances (2-norm of the difference over that of the result).  u = 2^-8 for
bf16, 2^-11 for fp16 (8 and 11 significant bits) is the largest relative error
of one rounding, its root mean square over a tensor about 0.43 u.
- o: the output rounding and up to four 16-bit operands (state, corrected
  values, scores, inverse) in sequence: sqrt(5) 0.43 u < 1.25 u.
- states: float32 to about 16 bits per product: 2e-5.
- gradients: up to eight 16-bit operands in sequence and the output's: 3 x
  0.43 u < 1.5 u; a gradient of a gate is a difference of such sums, which
  doubles it.
"""
import ctypes

import pytest
import torch

import fft_long_convolution_gb300 as F
from _mixers import delta_inputs, delta_rule, rel

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
DTYPES = [torch.bfloat16, torch.float16]
TOL_STATE = 2e-5


def tol_o(dt):
    return 1.25 * U[dt]


def tol_grad(dt, name):
    return (3 if name in ("dg", "dbeta") else 1.5) * U[dt]


def cuda(*xs):
    return [None if x is None else x.cuda() for x in xs]


def states(n, Hv, Dk, Dv, seed=9):
    gen = torch.Generator().manual_seed(seed)
    return 0.3 * torch.randn(n, Hv, Dk, Dv, generator=gen)


SIZES = [(1, 1, 1, 1, 64, 64), (2, 63, 2, 2, 64, 128), (1, 64, 1, 2, 128, 64), (3, 65, 2, 2, 128, 128),
         (2, 200, 1, 3, 64, 64), (1, 513, 2, 4, 128, 128), (5, 2, 3, 3, 64, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("B,T,Hk,Hv,Dk,Dv", SIZES)
@pytest.mark.parametrize("init", [False, True])
def test_forward(B, T, Hk, Hv, Dk, Dv, dt, init):
    ins = delta_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=T)
    s0 = states(B, Hv, Dk, Dv) if init else None
    ref, sref = delta_rule(*ins, state=s0, scale=Dk ** -0.5)
    plan = F.DeltaRule(Dk, Dv, dt)
    o, s = plan.forward(*cuda(*ins), state=None if s0 is None else s0.cuda())
    assert o.dtype == dt and s.dtype == torch.float32
    assert rel(o, ref) < tol_o(dt) and rel(s, sref) < TOL_STATE
    assert plan.device_status() == 0


def grads(ins, do, s0, ds, scale):
    xs = [x.double().requires_grad_() for x in ins]
    s = s0.double().requires_grad_()
    o, sT = delta_rule(*xs, state=s, scale=scale)
    loss = (o * do.double()).sum() + (sT * ds.double()).sum()
    return torch.autograd.grad(loss, xs + [s])


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("B,T,Hk,Hv,Dk,Dv", SIZES)
def test_backward(B, T, Hk, Hv, Dk, Dv, dt):
    ins = delta_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=T + 1)
    s0, ds = states(B, Hv, Dk, Dv), states(B, Hv, Dk, Dv, seed=10)
    do = delta_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=T + 2)[2]
    ref = grads(ins, do, s0, ds, Dk ** -0.5)
    plan = F.DeltaRule(Dk, Dv, dt)
    dins = cuda(*ins)
    _, _, saved = plan.forward(*dins, state=s0.cuda(), save=True)
    got = plan.backward(do.cuda(), *dins, saved, dstate=ds.cuda())
    for name, x, r in zip(("dq", "dk", "dv", "dg", "dbeta", "dstate"), got, ref):
        assert rel(x, r) < tol_grad(dt, name), name
    # without a gradient of the final states
    ref = grads(ins, do, s0, torch.zeros_like(ds), Dk ** -0.5)
    got = plan.backward(do.cuda(), *dins, saved)
    for name, x, r in zip(("dq", "dk", "dv", "dg", "dbeta", "dstate"), got, ref):
        assert rel(x, r) < tol_grad(dt, name), name
    again = plan.backward(do.cuda(), *dins, saved)
    assert all(torch.equal(x, y) for x, y in zip(got, again))
    assert plan.device_status() == 0


@pytest.mark.gpu
def test_backward_against_differences():
    """Directional derivatives of the 64-bit definition by central differences
    (step 1e-4: truncation 1e-8, far below the gradient tolerance)."""
    dt, B, T, Hk, Hv, Dk, Dv = torch.float16, 1, 70, 1, 2, 64, 64
    ins = delta_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=3)
    do = delta_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=4)[2]
    plan = F.DeltaRule(Dk, Dv, dt)
    dins = cuda(*ins)
    _, _, saved = plan.forward(*dins, save=True)
    got = plan.backward(do.cuda(), *dins, saved)[:5]
    xs = [x.double() for x in ins]
    for i, (x, gx) in enumerate(zip(xs, got)):
        gx = gx.double().cpu()
        # along the gradient itself, where the derivative is its norm
        way = gx / gx.norm()
        h = 1e-4
        vals = []
        for sgn in (1, -1):
            ys = list(xs)
            ys[i] = x + sgn * h * way
            vals.append(float((delta_rule(*ys, scale=Dk ** -0.5)[0] * do.double()).sum()))
        slope = (vals[0] - vals[1]) / (2 * h)
        assert abs(slope - float(gx.norm())) < tol_grad(dt, "dg") * float(gx.norm()), i


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("lens", [[0], [1], [3, 0, 64, 1, 65, 130, 0, 7], [64, 64], [5, 200, 1]])
def test_ragged(lens, dt):
    """Packed sequences, empty ones among them, against each one by itself;
    tokens after the last sequence belong to none."""
    Hk, Hv, Dk, Dv, n = 1, 2, 64, 128, len(lens)
    T = sum(lens) + 5
    ins = delta_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=n)
    do = delta_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=n + 1)[2]
    s0, ds = states(n, Hv, Dk, Dv), states(n, Hv, Dk, Dv, seed=12)
    off = torch.zeros(n + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(torch.tensor(lens), 0)
    plan = F.DeltaRule(Dk, Dv, dt)
    dins = cuda(*ins)
    o, s, saved = plan.forward(*dins, state=s0.cuda(), offsets=off.cuda(), save=True)
    got = plan.backward(do.cuda(), *dins, saved, dstate=ds.cuda(), offsets=off.cuda())
    for i, L in enumerate(lens):
        at = slice(int(off[i]), int(off[i]) + L)
        part = [x[:, at] for x in ins]
        ref, sref = delta_rule(*part, state=s0[i:i + 1], scale=Dk ** -0.5)
        assert rel(o[:, at], ref) < tol_o(dt) and rel(s[i:i + 1], sref) < TOL_STATE
        if L == 0:
            assert torch.equal(s[i].cpu(), s0[i]) and torch.equal(got[5][i].cpu(), ds[i])
            continue
        r = grads(part, do[:, at], s0[i:i + 1], ds[i:i + 1], Dk ** -0.5)
        for name, x, y in zip(("dq", "dk", "dv", "dg", "dbeta"), got, r):
            assert rel(x[:, at], y) < tol_grad(dt, name), (name, i)
        assert rel(got[5][i:i + 1], r[5]) < tol_grad(dt, "dstate")
    assert all(not bool(x[:, sum(lens):].any()) for x in [o] + list(got[:5]))


@pytest.mark.gpu
def test_sequences_do_not_touch_each_other():
    """NaN and infinities in one packed sequence stay in it."""
    dt, Hk, Hv, Dk, Dv = torch.bfloat16, 2, 2, 128, 128
    lens = [70, 30, 90]
    T = sum(lens)
    ins = delta_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=5)
    off = torch.tensor([0, 70, 100, 190], dtype=torch.int32)
    bad = [x.clone() for x in ins]
    for x, w in zip(bad, (float("nan"), float("inf"), float("-inf"), float("nan"), float("inf"))):
        x[:, 70:100] = w
    plan = F.DeltaRule(Dk, Dv, dt)
    do = delta_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=6)[2]
    res = []
    for y in (ins, bad):
        y = cuda(*y)
        o, s, saved = plan.forward(*y, offsets=off.cuda(), save=True)
        res.append([o, s] + list(plan.backward(do.cuda(), *y, saved, offsets=off.cuda())))
    for j, (x, y) in enumerate(zip(*res)):
        if j in (1, 7):  # states
            assert torch.equal(x[0], y[0]) and torch.equal(x[2], y[2])
        else:
            assert torch.equal(x[:, :70], y[:, :70]) and torch.equal(x[:, 100:], y[:, 100:])
    assert plan.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("low", [float("-inf"), "lowest", -200.0])
def test_resets(low, dt):
    """A log decay of -infinity (or the type's lowest value) empties the state:
    what follows is the sequence from there on."""
    B, T, Hk, Hv, Dk, Dv, at = 1, 150, 1, 1, 64, 64, 75
    ins = list(delta_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=7))
    low = torch.finfo(dt).min if low == "lowest" else low
    ins[3][:, at] = low
    ins[3][:, 0] = low
    do = delta_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=8)[2]
    s0 = states(B, Hv, Dk, Dv)
    plan = F.DeltaRule(Dk, Dv, dt)
    dins = cuda(*ins)
    o, s, saved = plan.forward(*dins, state=s0.cuda(), save=True)
    ref, sref = delta_rule(*[x[:, at:] for x in ins], scale=Dk ** -0.5)
    assert rel(o[:, at:], ref) < tol_o(dt) and rel(s, sref) < TOL_STATE
    got = plan.backward(do.cuda(), *dins, saved)
    fin = [x.clone() for x in ins]
    fin[3] = fin[3].double().clamp(min=-200.0)
    r = grads(fin, do, s0, torch.zeros_like(s0), Dk ** -0.5)
    for name, x, y in zip(("dq", "dk", "dv", "dg", "dbeta"), got, r):
        assert rel(x, y) < tol_grad(dt, name), name
    assert not bool(got[5].any()) and float(got[3][0, at, 0]) == 0.0


@pytest.mark.gpu
def test_strong_and_weak_decays():
    """Decays from none to e^-3 a token in one chunk: ratios of decays inside
    a chunk span e^-190 without overflow."""
    dt, B, T, Hk, Hv, Dk, Dv = torch.float16, 1, 192, 1, 3, 64, 64
    ins = list(delta_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=11))
    ins[3][:, :, 0], ins[3][:, :, 1] = 0.0, -3.0
    do = delta_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=12)[2]
    s0 = states(B, Hv, Dk, Dv)
    plan = F.DeltaRule(Dk, Dv, dt)
    dins = cuda(*ins)
    o, s, saved = plan.forward(*dins, state=s0.cuda(), save=True)
    ref, sref = delta_rule(*ins, state=s0, scale=Dk ** -0.5)
    for h in range(Hv):
        assert rel(o[:, :, h], ref[:, :, h]) < tol_o(dt) and rel(s[:, h], sref[:, h]) < TOL_STATE
    got = plan.backward(do.cuda(), *dins, saved)
    r = grads(ins, do, s0, torch.zeros_like(s0), Dk ** -0.5)
    for name, x, y in zip(("dq", "dk", "dv", "dg", "dbeta"), got, r):
        assert rel(x, y) < tol_grad(dt, name), name


@pytest.mark.gpu
def test_equal_keys_and_zero_gates():
    """All keys of a chunk equal (the triangular system at its stiffest), beta
    = 1; and beta = 0, where only decays act."""
    dt, B, T, Hk, Hv, Dk, Dv = torch.bfloat16, 1, 130, 1, 2, 128, 128
    q, k, v, g, beta = delta_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=13)
    k = torch.zeros_like(k)
    k[..., 0] = 1.0
    g = torch.zeros_like(g)
    beta = torch.ones_like(beta)
    beta[:, :, 1] = 0.0
    s0 = states(B, Hv, Dk, Dv)
    plan = F.DeltaRule(Dk, Dv, dt)
    dins = cuda(q, k, v, g, beta)
    o, s, saved = plan.forward(*dins, state=s0.cuda(), save=True)
    ref, sref = delta_rule(q, k, v, g, beta, state=s0, scale=Dk ** -0.5)
    assert rel(o, ref) < tol_o(dt) and rel(s, sref) < TOL_STATE
    do = v.flip(1).contiguous()
    got = plan.backward(do.cuda(), *dins, saved)
    r = grads((q, k, v, g, beta), do, s0, torch.zeros_like(s0), Dk ** -0.5)
    for name, x, y in zip(("dq", "dk", "dv", "dbeta"), [got[i] for i in (0, 1, 2, 4)], [r[i] for i in (0, 1, 2, 4)]):
        assert rel(x, y) < tol_grad(dt, name), name


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("B,T,Hk,Hv,Dk,Dv", [(1, 1, 1, 1, 64, 64), (3, 1, 2, 4, 128, 128), (5, 4, 1, 2, 64, 128),
                                             (2, 9, 3, 3, 128, 64)])
def test_step(B, T, Hk, Hv, Dk, Dv, dt):
    """Rows against scattered states; a row without a slot; in place and not."""
    ins = delta_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=B)
    pool = states(B + 3, Hv, Dk, Dv)
    slots = torch.randperm(B + 3, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32)
    if B > 2:
        slots[1], slots[2] = -1, B + 3
    used = [b for b in range(B) if 0 <= slots[b] < B + 3]
    plan = F.DeltaRule(Dk, Dv, dt)
    dev = pool.cuda()
    out = torch.full_like(dev, 7.0)
    dins = cuda(*ins)
    o = plan.step(*dins, dev, state_out=out, slots=slots.cuda())
    assert torch.equal(dev.cpu(), pool)
    o2 = plan.step(*dins, dev, slots=slots.cuda())
    assert torch.equal(o, o2)
    want = pool.clone()
    for b in range(B):
        if b not in used:
            assert not bool(o[b].any())
            continue
        ref, sref = delta_rule(*[x[b:b + 1] for x in ins], state=pool[slots[b]][None], scale=Dk ** -0.5)
        # float32 sums and one rounding of o
        assert rel(o[b:b + 1], ref) < U[dt]
        assert rel(dev[slots[b]][None], sref) < 1e-6
        assert torch.equal(out[slots[b]], dev[slots[b]])
        want[slots[b]] = dev[slots[b]].cpu()
    assert torch.equal(dev.cpu(), want)
    idle = [i for i in range(B + 3) if i not in [int(slots[b]) for b in used]]
    assert bool((out[idle] == 7.0).all())


@pytest.mark.gpu
def test_chunked_and_recurrent_agree():
    """A prompt, then tokens one by one, against the whole sequence."""
    dt, B, T, n, Hk, Hv, Dk, Dv = torch.float16, 2, 100, 4, 2, 2, 128, 64
    ins = delta_inputs(B, T + n, Hk, Hv, Dk, Dv, dt, seed=21)
    ref, sref = delta_rule(*ins, scale=Dk ** -0.5)
    plan = F.DeltaRule(Dk, Dv, dt)
    dins = cuda(*ins)
    _, s = plan.forward(*[x[:, :T] for x in dins])
    for t in range(T, T + n):
        o = plan.step(*[x[:, t:t + 1] for x in dins], s)
        assert rel(o, ref[:, t:t + 1]) < tol_o(dt)
    assert rel(s, sref) < TOL_STATE


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["fused", "head-major", "reversed-batch-layout"])
def test_strides_and_streams(order):
    """Slices of one projection, [B, H, T, D] and [T, B, H, D] storage, on a
    side stream: the results of contiguous tensors on the default stream."""
    dt, B, T, Hk, Hv, Dk, Dv = torch.bfloat16, 2, 130, 2, 4, 64, 128
    ins = delta_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=31)
    q, k, v, g, beta = cuda(*ins)
    plan = F.DeltaRule(Dk, Dv, dt)
    do = torch.flip(v, [1]).contiguous()
    o0, s0, saved = plan.forward(q, k, v, g, beta, save=True)
    g0 = plan.backward(do, q, k, v, g, beta, saved)
    if order == "fused":
        flat = torch.cat([x.flatten(2) for x in (q, k, v)], -1)
        q, k, v = (x.unflatten(2, s) for x, s in zip(flat.split([Hk * Dk, Hk * Dk, Hv * Dv], -1),
                                                     ((Hk, Dk), (Hk, Dk), (Hv, Dv))))
        gb = torch.stack([g, beta], -1)
        g, beta = gb[..., 0], gb[..., 1]
    else:
        way = (lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)) if order == "head-major" else \
            (lambda x: x.transpose(0, 1).contiguous().transpose(0, 1))
        q, k, v, g, beta, do = (way(x) for x in (q, k, v, g, beta, do))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o1, s1, saved = plan.forward(q, k, v, g, beta, save=True, stream=side)
    g1 = plan.backward(do, q, k, v, g, beta, saved, stream=side)
    side.synchronize()
    assert torch.equal(o0, o1) and torch.equal(s0, s1)
    assert all(torch.equal(x, y) for x, y in zip(g0, g1))


@pytest.mark.gpu
def test_empty_calls():
    dt = torch.bfloat16
    plan = F.DeltaRule(64, 64, dt)
    s0 = states(2, 1, 64, 64).cuda()
    ins = cuda(*delta_inputs(2, 0, 1, 1, 64, 64, dt))
    o, s = plan.forward(*ins, state=s0)
    assert o.shape == (2, 0, 1, 64) and torch.equal(s, s0)
    assert not bool(plan.forward(*ins)[1].any())
    ins = cuda(*delta_inputs(0, 5, 1, 1, 64, 64, dt))
    o, s = plan.forward(*ins)
    assert o.shape == (0, 5, 1, 64) and s.shape[0] == 0


@pytest.mark.gpu
def test_offsets_outside_the_row_are_clamped():
    dt, Hk, Hv, Dk, Dv, T = torch.bfloat16, 1, 1, 64, 64, 80
    ins = delta_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=41)
    plan = F.DeltaRule(Dk, Dv, dt)
    off = torch.tensor([-5, 30, 20, 1000], dtype=torch.int32).cuda()  # [0, 30), empty, [20, 80)
    o, s = plan.forward(*cuda(*ins), offsets=off)
    torch.cuda.synchronize()
    ref, sref = delta_rule(*[x[:, :30] for x in ins], scale=Dk ** -0.5)
    assert rel(s[:1], sref) < TOL_STATE and not bool(s[1].any())
    ref, sref = delta_rule(*[x[:, 20:] for x in ins], scale=Dk ** -0.5)
    assert rel(s[2:], sref) < TOL_STATE


@pytest.mark.gpu
def test_no_sequences_and_tokens_before_the_first():
    """A packed row without sequences is all zeros; so are tokens before the
    first sequence."""
    dt, Hk, Hv, Dk, Dv, T = torch.float16, 1, 2, 64, 64, 90
    ins = cuda(*delta_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=42))
    plan = F.DeltaRule(Dk, Dv, dt)
    for off in ([0], [20, 50]):
        off = torch.tensor(off, dtype=torch.int32).cuda()
        torch.full((1, T, Hv, Dv), 3.0, dtype=dt, device="cuda")  # what the allocator hands out next is not zero
        o, s, saved = plan.forward(*ins, offsets=off, save=True)
        got = plan.backward(ins[2], *ins, saved, offsets=off)
        live = torch.zeros(T, dtype=torch.bool)
        if off.numel() > 1:
            live[20:50] = True
            ref, sref = delta_rule(*[x.cpu()[:, 20:50] for x in ins], scale=Dk ** -0.5)
            assert rel(o[:, 20:50], ref) < tol_o(dt) and rel(s, sref) < TOL_STATE
        for x in [o] + list(got[:5]):
            assert not bool(x.cpu()[:, ~live].any())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("B,T,Hk,Hv,Dk,Dv", [(1, 12000, 1, 1, 64, 64), (1, 8200, 1, 2, 128, 64), (2, 6500, 1, 1, 64, 128)])
def test_long_rows_in_segments(B, T, Hk, Hv, Dk, Dv, dt):
    """Rows long and few enough to be cut into segments, with and without an
    initial state; compared at the end and on a sample of the outputs, so that
    the 64-bit side stays small."""
    ins = delta_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=51)
    s0 = states(B, Hv, Dk, Dv)
    plan = F.DeltaRule(Dk, Dv, dt)
    ref, sref = delta_rule(*ins, state=s0, scale=Dk ** -0.5)
    o, s = plan.forward(*cuda(*ins), state=s0.cuda())
    assert rel(o, ref) < tol_o(dt) and rel(s, sref) < TOL_STATE
    assert plan.device_status() == 0


@pytest.mark.gpu
def test_refusals():
    dt = torch.bfloat16
    B, T, Hk, Hv, Dk, Dv = 2, 70, 1, 2, 64, 64
    q, k, v, g, beta = cuda(*delta_inputs(B, T, Hk, Hv, Dk, Dv, dt))
    plan = F.DeltaRule(Dk, Dv, dt)

    def status(f):
        with pytest.raises(F.FFTConvError) as e:
            f()
        return e.value.status

    with pytest.raises(ValueError):
        plan.forward(q.float(), k, v, g, beta)
    with pytest.raises(ValueError):
        plan.forward(q, k, v, g[:, :-1], beta)
    with pytest.raises(ValueError):
        plan.forward(q, k, v, g, beta, state=torch.zeros(B, Hv, Dk, Dv))
    with pytest.raises(ValueError):
        plan.forward(q, k, v.transpose(2, 3).contiguous().transpose(2, 3), g, beta)
    # heads that do not divide
    assert status(lambda: plan.forward(torch.cat([q] * 3, 2), torch.cat([k] * 3, 2), v, g, beta)) == 1
    # a row that starts off a 16-byte boundary; a token stride that is not a multiple of 8
    wide = torch.zeros(B, T, Hk, Dk + 8, dtype=dt, device="cuda")
    assert status(lambda: plan.forward(wide[..., 4:4 + Dk], k, v, g, beta)) == 3
    odd = torch.zeros(B, T, Hk * Dk + 4, dtype=dt, device="cuda")[..., :Dk].unflatten(2, (1, Dk))
    assert status(lambda: plan.forward(odd, k, v, g, beta)) == 3
    # a broadcast batch has stride 0
    assert status(lambda: plan.forward(q[:1].expand(B, -1, -1, -1), k, v, g, beta)) == 1
    # offsets with more than one row
    off = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    assert status(lambda: plan.forward(q, k, v, g, beta, offsets=off)) == 1
    # outputs over inputs
    L = F.lib()
    a = plan._args(q, k, v, g, beta, None, None)
    vo = F.View(*F._strides(v, "v", dt, v.shape))
    need = L.fftconv_delta_scratch_bytes(plan._h, B, T, Hk, Hv, B, 0)
    scratch = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    assert L.fftconv_delta_forward(plan._h, ctypes.byref(a), None, vo, None, None, scratch.data_ptr(), need, None) == 1
    o = torch.empty_like(v)
    ov = F.View(*F._strides(o, "o", dt, o.shape))
    if need:
        assert L.fftconv_delta_forward(plan._h, ctypes.byref(a), None, ov, None, None, None, 0, None) == 4
    assert L.fftconv_delta_backward(plan._h, ctypes.byref(a), ov, None, None, ov, ov, ov, ov, ov, None, None, 0, None) == 1
    pool = torch.zeros(B - 1, Hv, Dk, Dv, device="cuda")
    assert status(lambda: plan.step(q[:, :1], k[:, :1], v[:, :1], g[:, :1], beta[:, :1], pool)) == 1
    big = torch.zeros(B + 1, Hv, Dk, Dv, device="cuda")
    assert status(lambda: plan.step(q[:, :1], k[:, :1], v[:, :1], g[:, :1], beta[:, :1], big[:-1], state_out=big[1:])) == 1


def test_refusals_without_gpu():
    L = F.lib()
    h = ctypes.c_void_p()
    for dk, dv, dt in ((32, 64, 1), (64, 256, 1), (0, 64, 0), (64, 64, 5)):
        assert L.fftconv_delta_create(ctypes.byref(h), dk, dv, dt) == 2 and not h.value
    assert L.fftconv_delta_create(None, 64, 64, 0) == 1
    assert L.fftconv_delta_destroy(None) == 0
    assert L.fftconv_delta_saved_bytes(None, 1, 1, 1, 1) == 0
    assert L.fftconv_delta_scratch_bytes(None, 1, 1, 1, 1, 1, 1) == 0
    a, view = F.DeltaArgs(), F.View(None, 0, 0, 0)
    assert L.fftconv_delta_forward(None, ctypes.byref(a), None, view, None, None, None, 0, None) == 1
    assert L.fftconv_delta_step(None, ctypes.byref(a), None, None, 0, None, view, None) == 1
    assert L.fftconv_delta_status(None, None, None) == 1
