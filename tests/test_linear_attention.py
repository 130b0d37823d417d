"""Linear attention with a decay for each head on the GPU against its 64-bit
definition.

Tolerances (2-norm of the difference over that of the result).
- o and the gradients in 16 bits: u = 2^-8 for bf16, 2^-11 for fp16 is the largest
  error of one rounding, its root mean square about 0.43 u; the result is rounded at
  the end, and of its two terms each has one operand rounded to 16 bits (the state;
  the scores): sqrt(3) 0.43 u = 0.75 u if the terms are as large as the result.  So u
  holds them.
- states and their gradients: float32 sums; an addition into a tensor-core
  accumulator may cut instead of round (2^-23), at most 12 of them a chunk of 64
  tokens, and one for every chunk after it: (12 + 9) 2^-23 < 3e-6 for rows of up
  to 9 chunks, with the parts' 2^-22 4e-6.
"""
import ctypes

import pytest
import torch

import fft_long_convolution_gb300 as F
from _attention import attention_grads, attention_inputs, linear_attention, rel, states

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
DTYPES = [torch.bfloat16, torch.float16]
TOL_STATE = 4e-6
NAMES = ("dq", "dk", "dv", "dstate")


def tol(name, dt):
    return TOL_STATE if name == "dstate" else U[dt]


def cuda(*xs):
    return [None if x is None else x.cuda() for x in xs]


SIZES = [(1, 1, 1, 1, 64, 64), (2, 63, 2, 2, 64, 128), (1, 64, 1, 2, 128, 64), (3, 65, 2, 2, 128, 128),
         (2, 200, 1, 3, 64, 64), (1, 513, 2, 4, 128, 128), (5, 2, 3, 3, 64, 64), (1, 128, 1, 1, 128, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("B,T,Hk,Hv,Dk,Dv", SIZES)
@pytest.mark.parametrize("init", [False, True])
def test_forward(B, T, Hk, Hv, Dk, Dv, dt, init):
    ins = attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=T)
    s0 = states(B, Hv, Dk, Dv) if init else None
    ref, sref = linear_attention(*ins, state=s0, scale=Dk ** -0.5)
    plan = F.LinearAttention(Dk, Dv, dt)
    o, s = plan.forward(*cuda(*ins), state=None if s0 is None else s0.cuda())
    assert o.dtype == dt and s.dtype == torch.float32
    assert rel(o, ref) < U[dt] and rel(s, sref) < TOL_STATE
    assert plan.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("B,T,Hk,Hv,Dk,Dv", SIZES)
def test_backward(B, T, Hk, Hv, Dk, Dv, dt):
    ins = attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=T + 1)
    s0, ds = states(B, Hv, Dk, Dv), states(B, Hv, Dk, Dv, seed=10)
    do = attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=T + 2)[2]
    plan = F.LinearAttention(Dk, Dv, dt)
    dins = cuda(*ins)
    for a, b in ((s0, ds), (None, None)):
        ref = attention_grads(*ins, do, torch.zeros_like(s0) if a is None else a, torch.zeros_like(ds) if b is None else b, Dk ** -0.5)
        got = plan.backward(do.cuda(), *dins, state=None if a is None else a.cuda(), dstate=None if b is None else b.cuda())
        for name, x, r in zip(NAMES, got, ref):
            assert (x is None and a is None and name == "dstate") or rel(x, r) < tol(name, dt), name
        again = plan.backward(do.cuda(), *dins, state=None if a is None else a.cuda(), dstate=None if b is None else b.cuda())
        assert all(x is y is None or torch.equal(x, y) for x, y in zip(got, again))
    assert plan.device_status() == 0


@pytest.mark.gpu
def test_backward_against_differences():
    """Directional derivatives of the 64-bit definition by central differences
    (the definition is linear along each of these inputs: no truncation)."""
    dt, B, T, Hk, Hv, Dk, Dv = torch.float16, 1, 70, 1, 2, 64, 64
    ins = attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=3)
    do = attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=4)[2]
    s0 = states(B, Hv, Dk, Dv)
    plan = F.LinearAttention(Dk, Dv, dt)
    got = plan.backward(do.cuda(), *cuda(*ins), state=s0.cuda())
    xs = [x.double() for x in (*ins[:3], s0)]
    for i, (x, gx) in enumerate(zip(xs, got)):
        gx = gx.double().cpu()
        way = gx / gx.norm()  # along the gradient itself, where the derivative is its norm
        vals = []
        for sgn in (1, -1):
            ys = list(xs)
            ys[i] = x + sgn * 1e-3 * way
            vals.append(float((linear_attention(*ys[:3], ins[3], ys[3], Dk ** -0.5)[0] * do.double()).sum()))
        slope = (vals[0] - vals[1]) / 2e-3
        assert abs(slope - float(gx.norm())) < U[dt] * float(gx.norm()), i


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("lens", [[0], [1], [3, 0, 64, 1, 65, 130, 0, 7], [64, 64], [5, 200, 1]])
@pytest.mark.parametrize("before", [0, 9])
def test_ragged(lens, before, dt):
    """Packed sequences, empty ones among them, against each one by itself; tokens
    before the first sequence and after the last one belong to none."""
    Hk, Hv, Dk, Dv, n = 1, 2, 64, 128, len(lens)
    T = before + sum(lens) + 5
    ins = attention_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=n)
    do = attention_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=n + 1)[2]
    s0, ds = states(n, Hv, Dk, Dv), states(n, Hv, Dk, Dv, seed=12)
    off = torch.full((n + 1,), before, dtype=torch.int32)
    off[1:] += torch.cumsum(torch.tensor(lens), 0)
    plan = F.LinearAttention(Dk, Dv, dt)
    dins = cuda(*ins)
    torch.full((1, T, Hv, Dv), 3.0, dtype=dt, device="cuda")  # what the allocator hands out next is not zero
    o, s = plan.forward(*dins, state=s0.cuda(), offsets=off.cuda())
    got = plan.backward(do.cuda(), *dins, state=s0.cuda(), dstate=ds.cuda(), offsets=off.cuda())
    live = torch.zeros(T, dtype=torch.bool)
    for i, L in enumerate(lens):
        at = slice(int(off[i]), int(off[i]) + L)
        live[at] = True
        part = [x[:, at] for x in ins[:3]] + [ins[3]]
        ref, sref = linear_attention(*part, state=s0[i:i + 1], scale=Dk ** -0.5)
        assert rel(o[:, at], ref) < U[dt] and rel(s[i:i + 1], sref) < TOL_STATE
        if L == 0:
            assert torch.equal(s[i].cpu(), s0[i]) and torch.equal(got[3][i].cpu(), ds[i])
            continue
        r = attention_grads(*part, do[:, at], s0[i:i + 1], ds[i:i + 1], Dk ** -0.5)
        for name, x, y in zip(NAMES[:3], got, r):
            assert rel(x[:, at], y) < tol(name, dt), (name, i)
        assert rel(got[3][i:i + 1], r[3]) < TOL_STATE
    for x in [o] + list(got[:3]):
        assert not bool(x.cpu()[:, ~live].any())
    assert plan.device_status() == 0


@pytest.mark.gpu
def test_sequences_and_heads_do_not_touch_each_other():
    """NaN and infinities in one packed sequence stay in it, a NaN decay in its head."""
    dt, Hk, Hv, Dk, Dv = torch.bfloat16, 2, 2, 128, 128
    T = 190
    ins = attention_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=5)
    off = torch.tensor([0, 70, 100, 190], dtype=torch.int32).cuda()
    do = attention_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=6)[2]
    s0 = states(3, Hv, Dk, Dv).cuda()
    bad = [x.clone() for x in ins]
    for x, w in zip(bad[:3], (float("nan"), float("inf"), float("-inf"))):
        x[:, 70:100] = w
    plan = F.LinearAttention(Dk, Dv, dt)

    def run(y):
        y = cuda(*y)
        return [*plan.forward(*y, state=s0, offsets=off), *plan.backward(do.cuda(), *y, state=s0, offsets=off)]

    good = run(ins)
    for j, (x, y) in enumerate(zip(good, run(bad))):
        if j in (1, 5):  # states
            assert torch.equal(x[0], y[0]) and torch.equal(x[2], y[2]), j
        else:
            assert torch.equal(x[:, :70], y[:, :70]) and torch.equal(x[:, 100:], y[:, 100:]), j
    lost = ins[3].clone()
    lost[1] = float("nan")
    for j, (x, y) in enumerate(zip(good, run([*ins[:3], lost]))):
        if j in (1, 5):
            assert torch.equal(x[:, 0], y[:, 0]) and bool(y[:, 1].isnan().any())
        else:
            assert torch.equal(x[:, :, 0], y[:, :, 0]) and bool(y[:, :, 1].isnan().any())
    assert plan.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
def test_decays_from_none_to_resets(dt):
    """Heads that keep everything, almost everything, little and nothing, and a
    decay above 0, which counts as 0; each head against its own definition."""
    B, T, Hk, Dk, Dv = 2, 200, 1, 64, 64
    logs = [0.0, -1e-6, -0.01, -0.7, -3.0, -50.0, -119.0, -200.0, torch.finfo(torch.float32).min, float("-inf"), 1.0]
    Hv = len(logs)
    q, k, v, _ = attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=11)
    decay = torch.tensor(logs)
    do = attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=12)[2]
    s0, ds = states(B, Hv, Dk, Dv), states(B, Hv, Dk, Dv, seed=13)
    plan = F.LinearAttention(Dk, Dv, dt)
    dins = cuda(q, k, v, decay)
    o, s = plan.forward(*dins, state=s0.cuda())
    got = plan.backward(do.cuda(), *dins, state=s0.cuda(), dstate=ds.cuda())
    ref, sref = linear_attention(q, k, v, decay, s0, Dk ** -0.5)
    r = attention_grads(q, k, v, decay, do, s0, ds, Dk ** -0.5)
    for h in range(Hv):
        assert rel(o[:, :, h], ref[:, :, h]) < U[dt] and rel(s[:, h], sref[:, h]) < TOL_STATE, h
        assert rel(got[2][:, :, h], r[2][:, :, h]) < U[dt], h
        if float(r[3][:, h].norm()) > 1e-30:  # else below float32
            assert rel(got[3][:, h], r[3][:, h]) < TOL_STATE, h
        else:
            assert float(got[3][:, h].norm()) < 1e-30
    for name, x, y in zip(NAMES[:2], got, r):  # sums over the heads
        assert rel(x, y) < U[dt], name
    step = torch.empty_like(s0).cuda()
    o1 = plan.step(*[x[:, :1] for x in dins[:3]], dins[3], s0.cuda(), state_out=step)
    ref, sref = linear_attention(q[:, :1], k[:, :1], v[:, :1], decay, s0, Dk ** -0.5)
    assert rel(o1, ref) < U[dt] and rel(step, sref) < 1e-6


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("B,T,Hk,Hv,Dk,Dv", [(1, 1, 1, 1, 64, 64), (3, 1, 2, 4, 128, 128), (5, 4, 1, 2, 64, 128),
                                             (2, 9, 3, 3, 128, 64)])
def test_step(B, T, Hk, Hv, Dk, Dv, dt):
    """Rows against scattered states; a row without a slot; in place and not."""
    ins = attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=B)
    pool = states(B + 3, Hv, Dk, Dv)
    slots = torch.randperm(B + 3, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32)
    if B > 2:
        slots[1], slots[2] = -1, B + 3
    used = [b for b in range(B) if 0 <= slots[b] < B + 3]
    plan = F.LinearAttention(Dk, Dv, dt)
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
        ref, sref = linear_attention(*[x[b:b + 1] for x in ins[:3]], ins[3], pool[slots[b]][None], Dk ** -0.5)
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
    ins = attention_inputs(B, T + n, Hk, Hv, Dk, Dv, dt, seed=21)
    ref, sref = linear_attention(*ins, scale=Dk ** -0.5)
    plan = F.LinearAttention(Dk, Dv, dt)
    dins = cuda(*ins)
    _, s = plan.forward(*[x[:, :T] for x in dins[:3]], dins[3])
    for t in range(T, T + n):
        o = plan.step(*[x[:, t:t + 1] for x in dins[:3]], dins[3], s)
        assert rel(o, ref[:, t:t + 1]) < U[dt]
    assert rel(s, sref) < TOL_STATE


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["fused", "head-major", "token-major-batch"])
def test_strides_and_streams(order):
    """Slices of one projection, [B, H, T, D] and [T, B, H, D] storage, on a
    side stream: the results of contiguous tensors on the default stream."""
    dt, B, T, Hk, Hv, Dk, Dv = torch.bfloat16, 2, 130, 2, 4, 64, 128
    q, k, v, decay = cuda(*attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=31))
    plan = F.LinearAttention(Dk, Dv, dt)
    do = torch.flip(v, [1]).contiguous()
    o0, s0 = plan.forward(q, k, v, decay)
    g0 = plan.backward(do, q, k, v, decay)
    if order == "fused":
        flat = torch.cat([x.flatten(2) for x in (q, k, v)], -1)
        q, k, v = (x.unflatten(2, s) for x, s in zip(flat.split([Hk * Dk, Hk * Dk, Hv * Dv], -1), ((Hk, Dk), (Hk, Dk), (Hv, Dv))))
    else:
        way = (lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)) if order == "head-major" else \
            (lambda x: x.transpose(0, 1).contiguous().transpose(0, 1))
        q, k, v, do = (way(x) for x in (q, k, v, do))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o1, s1 = plan.forward(q, k, v, decay, stream=side)
    g1 = plan.backward(do, q, k, v, decay, stream=side)
    side.synchronize()
    assert torch.equal(o0, o1) and torch.equal(s0, s1)
    assert all(torch.equal(x, y) for x, y in zip(g0[:3], g1[:3]))


@pytest.mark.gpu
def test_empty_calls():
    dt = torch.bfloat16
    plan = F.LinearAttention(64, 64, dt)
    s0 = states(2, 1, 64, 64).cuda()
    ins = cuda(*attention_inputs(2, 0, 1, 1, 64, 64, dt))
    o, s = plan.forward(*ins, state=s0)
    assert o.shape == (2, 0, 1, 64) and torch.equal(s, s0)
    assert not bool(plan.forward(*ins)[1].any())
    assert torch.equal(plan.backward(ins[2], *ins, state=s0, dstate=s0)[3], s0)
    ins = cuda(*attention_inputs(0, 5, 1, 1, 64, 64, dt))
    o, s = plan.forward(*ins)
    assert o.shape == (0, 5, 1, 64) and s.shape[0] == 0
    q = torch.ones(2, 5, 3, 64, dtype=dt, device="cuda")
    none = torch.empty(2, 5, 0, 64, dtype=dt, device="cuda")
    dq, dk, dv, _ = plan.backward(none, q, q, none, torch.empty(0, device="cuda"))
    assert not bool(dq.any()) and not bool(dk.any()) and dv.numel() == 0


@pytest.mark.gpu
def test_offsets_outside_the_row_are_clamped_and_no_sequences():
    dt, Hk, Hv, Dk, Dv, T = torch.bfloat16, 1, 1, 64, 64, 80
    ins = attention_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=41)
    plan = F.LinearAttention(Dk, Dv, dt)
    off = torch.tensor([-5, 30, 20, 1000], dtype=torch.int32).cuda()  # [0, 30), empty, [20, 80)
    o, s = plan.forward(*cuda(*ins), offsets=off)
    torch.cuda.synchronize()
    _, sref = linear_attention(*[x[:, :30] for x in ins[:3]], ins[3])
    assert rel(s[:1], sref) < TOL_STATE and not bool(s[1].any())
    _, sref = linear_attention(*[x[:, 20:] for x in ins[:3]], ins[3])
    assert rel(s[2:], sref) < TOL_STATE
    torch.full((1, T, Hv, Dv), 3.0, dtype=dt, device="cuda")
    o, s = plan.forward(*cuda(*ins), offsets=off[:1])
    got = plan.backward(ins[2].cuda(), *cuda(*ins), offsets=off[:1])
    assert s.shape[0] == 0 and not any(bool(x.any()) for x in (o, *got[:3]))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("B,T,Hk,Hv,Dk,Dv", [(1, 6000, 1, 1, 64, 64), (1, 4111, 1, 2, 128, 64), (2, 3300, 1, 1, 64, 128),
                                             (1, 5001, 1, 1, 128, 128)])
def test_long_rows(B, T, Hk, Hv, Dk, Dv, dt):
    """Rows long and few enough to be cut into segments.  Up to 94 chunks: (12 +
    94) 2^-23 = 1.3e-5 for the states."""
    ins = attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=51)
    ins[3][0] = 0.0
    s0, ds = states(B, Hv, Dk, Dv), states(B, Hv, Dk, Dv, seed=52)
    do = attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=53)[2]
    plan = F.LinearAttention(Dk, Dv, dt)
    ref, sref = linear_attention(*ins, state=s0, scale=Dk ** -0.5)
    dins = cuda(*ins)
    o, s = plan.forward(*dins, state=s0.cuda())
    assert rel(o, ref) < U[dt] and rel(s, sref) < 1.3e-5
    got = plan.backward(do.cuda(), *dins, state=s0.cuda(), dstate=ds.cuda())
    r = attention_grads(*ins, do, s0, ds, Dk ** -0.5)
    for name, x, y in zip(NAMES, got, r):
        assert rel(x, y) < (1.3e-5 if name == "dstate" else U[dt]), name
    assert plan.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
def test_uneven_queue(dt):
    """One long prompt among short ones, all packed into one row."""
    Hk, Hv, Dk, Dv = 1, 1, 64, 64
    lens = [40, 3000, 1, 0, 70, 64, 900]
    T, n = sum(lens), len(lens)
    ins = attention_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=61)
    do = attention_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=62)[2]
    s0, ds = states(n, Hv, Dk, Dv), states(n, Hv, Dk, Dv, seed=63)
    off = torch.zeros(n + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(torch.tensor(lens), 0)
    plan = F.LinearAttention(Dk, Dv, dt)
    dins = cuda(*ins)
    o, s = plan.forward(*dins, state=s0.cuda(), offsets=off.cuda())
    got = plan.backward(do.cuda(), *dins, state=s0.cuda(), dstate=ds.cuda(), offsets=off.cuda())
    for i, L in enumerate(lens):
        at = slice(int(off[i]), int(off[i]) + L)
        part = [x[:, at] for x in ins[:3]] + [ins[3]]
        ref, sref = linear_attention(*part, state=s0[i:i + 1], scale=Dk ** -0.5)
        assert rel(o[:, at], ref) < U[dt] and rel(s[i:i + 1], sref) < 8e-6  # (12 + 47) 2^-23
        if L:
            r = attention_grads(*part, do[:, at], s0[i:i + 1], ds[i:i + 1], Dk ** -0.5)
            for name, x, y in zip(NAMES[:3], got, r):
                assert rel(x[:, at], y) < U[dt], (name, i)
            assert rel(got[3][i:i + 1], r[3]) < 8e-6
    assert plan.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("size", [1e-3, 1.0, 300.0])
def test_fp16_values_of_other_sizes(size):
    """Values and given gradients far from 1 (a scaled or an unscaled loss): states
    and their gradients keep float32's digits, whatever 16 bits hold.  o, dq, dk, dv
    within u where they are normal numbers: below 2^-14 = 6.1e-5 a step is 2^-24, and
    the rounding at the end is off by up to 2^-25 an element.  Past 65504 (products of
    values and gradients of 300, summed: 1e6) a 16-bit result is an infinity; near there
    it may be either: the operands' roundings, 0.43 u of each term in root mean square,
    add up to 0.43 u sqrt(sum of squared terms), which for terms of either sign is
    0.43 u times the root mean square of the results, whatever one element's own size
    (that is 1e6 here, and 8 deviations of it 3.4 u)."""
    dt, B, T, Hk, Hv, Dk, Dv = torch.float16, 1, 300, 1, 1, 64, 128
    q, k, v, decay = attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=71)
    q = q * 0.1
    v = (v.double() * size).to(dt)
    do = (attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=72)[2].double() * size).to(dt)
    s0 = states(B, Hv, Dk, Dv) * size * 30
    plan = F.LinearAttention(Dk, Dv, dt)
    dins = cuda(q, k, v, decay)
    o, s = plan.forward(*dins, state=s0.cuda())
    ref, sref = linear_attention(q, k, v, decay, s0, Dk ** -0.5)

    def near(x, y):
        x, floor = x.double().cpu(), 2.0 ** -25 * y.numel() ** 0.5
        near_top = 65504 * 2.0 ** -9 + 4 * U[dt] * float(y.norm()) / y.numel() ** 0.5
        fits, huge = y.abs() < 65504 - near_top, y.abs() > 65504 + near_top
        return torch.equal(x[huge], y[huge].sign() * float("inf")) and \
            float((x - y)[fits].norm()) < U[dt] * float(y.norm()) + floor

    assert near(o, ref) and rel(s, sref) < TOL_STATE
    got = plan.backward(do.cuda(), *dins, state=s0.cuda())
    r = attention_grads(q, k, v, decay, do, s0, torch.zeros_like(s0), Dk ** -0.5)
    assert all(near(x, y) for x, y in zip(got[:3], r[:3])) and rel(got[3], r[3]) < TOL_STATE


@pytest.mark.gpu
def test_states_beyond_fp16():
    """States of 1e6, which 16-bit floats do not hold, against queries of 1e-3."""
    dt, B, T, Hk, Hv, Dk, Dv = torch.float16, 1, 130, 1, 1, 128, 64
    q, k, v, decay = attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=81)
    q = (q.double() * 1e-3).to(dt)
    s0 = states(B, Hv, Dk, Dv) * 1e6
    plan = F.LinearAttention(Dk, Dv, dt)
    o, s = plan.forward(*cuda(q, k, v, decay), state=s0.cuda())
    ref, sref = linear_attention(q, k, v, decay, s0, Dk ** -0.5)
    assert bool(o.isfinite().all()) and rel(o, ref) < U[dt] and rel(s, sref) < TOL_STATE


@pytest.mark.gpu
def test_captured_calls_replay():
    """A prompt, its gradients and a step captured into one graph and replayed on
    new inputs: the same bits as the calls."""
    dt, B, T, Hk, Hv, Dk, Dv = torch.bfloat16, 2, 150, 1, 2, 64, 64
    plan = F.LinearAttention(Dk, Dv, dt)
    first, second = (cuda(*attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=s)) for s in (91, 92))
    held = [x.clone() for x in first]

    def work(y):
        o, s = plan.forward(*y)
        g = plan.backward(y[2], *y, state=s, dstate=s)
        state = s.clone()
        return [o, s, *g, plan.step(*[x[:, :1] for x in y[:3]], y[3], state), state]

    work(held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = work(held)
    for ins in (first, second):
        for x, y in zip(held, ins):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(kept, work(ins)))


@pytest.mark.gpu
def test_two_streams_at_once():
    """One plan from two streams side by side: each call has its own workspace."""
    dt, B, T, Hk, Hv, Dk, Dv = torch.float16, 1, 5000, 1, 2, 64, 64
    plan = F.LinearAttention(Dk, Dv, dt)
    ins = [cuda(*attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=s)) for s in (101, 102)]
    want = [[*plan.forward(*x), *plan.backward(x[2], *x)[:3]] for x in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [[] for _ in ins]
    for _ in range(3):
        for i, (x, st) in enumerate(zip(ins, streams)):
            got[i] = [*plan.forward(*x, stream=st), *plan.backward(x[2], *x, stream=st)[:3]]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for a, b in zip(want, got) for x, y in zip(a, b))


@pytest.mark.gpu
def test_refusals():
    dt = torch.bfloat16
    B, T, Hk, Hv, Dk, Dv = 2, 70, 1, 2, 64, 64
    q, k, v, decay = cuda(*attention_inputs(B, T, Hk, Hv, Dk, Dv, dt))
    plan = F.LinearAttention(Dk, Dv, dt)

    def status(f):
        with pytest.raises(F.FFTConvError) as e:
            f()
        return e.value.status

    for bad in (lambda: plan.forward(q.float(), k, v, decay), lambda: plan.forward(q, k, v, decay[:1]),
                lambda: plan.forward(q, k, v, None), lambda: plan.forward(q, k, v, decay.double()),
                lambda: plan.forward(q, k, v, decay.cpu()),
                lambda: plan.forward(q, k, v, decay, state=torch.zeros(B, Hv, Dk, Dv)),
                lambda: plan.forward(q, k, v.transpose(2, 3).contiguous().transpose(2, 3), decay),
                lambda: plan.backward(v[:, 1:], q, k, v, decay)):
        with pytest.raises(ValueError):
            bad()
    # heads that do not divide
    assert status(lambda: plan.forward(torch.cat([q] * 3, 2), torch.cat([k] * 3, 2), v, decay)) == 1
    # a row that starts off a 16-byte boundary; a token stride that is not a multiple of 8
    wide = torch.zeros(B, T, Hk, Dk + 8, dtype=dt, device="cuda")
    assert status(lambda: plan.forward(wide[..., 4:4 + Dk], k, v, decay)) == 3
    odd = torch.zeros(B, T, Hk * Dk + 4, dtype=dt, device="cuda")[..., :Dk].unflatten(2, (1, Dk))
    assert status(lambda: plan.forward(odd, k, v, decay)) == 3
    # a broadcast batch has stride 0
    assert status(lambda: plan.forward(q[:1].expand(B, -1, -1, -1), k, v, decay)) == 1
    # offsets with more than one row
    off = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    assert status(lambda: plan.forward(q, k, v, decay, offsets=off)) == 1
    # outputs over inputs and over each other, missing scratch
    L = F.lib()
    a = plan._args(q, k, v, decay, None, None)
    vo = F.View(*F._strides(v, "v", dt, v.shape))
    o = torch.empty_like(v)
    ov = F.View(*F._strides(o, "o", dt, o.shape))
    need = [L.fftconv_linattn_scratch_bytes(plan._h, B, T, Hk, Hv, B, i) for i in (0, 1)]
    scratch = torch.empty(max(need + [16]), dtype=torch.uint8, device="cuda")
    assert L.fftconv_linattn_forward(plan._h, ctypes.byref(a), None, vo, None, scratch.data_ptr(), need[0], None) == 1
    assert L.fftconv_linattn_forward(plan._h, ctypes.byref(a), None, ov, o.data_ptr(), scratch.data_ptr(), need[0], None) == 1
    dq, dk = (F.View(*F._strides(torch.empty_like(q), "q", dt, q.shape)) for _ in range(2))
    assert need[1] and L.fftconv_linattn_backward(plan._h, ctypes.byref(a), None, vo, None, dq, dk, ov, None, None, 0, None) == 4
    assert L.fftconv_linattn_backward(plan._h, ctypes.byref(a), None, vo, None, dq, dk, vo, None, scratch.data_ptr(), need[1], None) == 1
    assert L.fftconv_linattn_backward(plan._h, ctypes.byref(a), None, vo, None, dq, dk, ov, o.data_ptr(), scratch.data_ptr(),
                                      need[1], None) == 1
    pool = torch.zeros(B - 1, Hv, Dk, Dv, device="cuda")
    one = [x[:, :1] for x in (q, k, v)]
    assert status(lambda: plan.step(*one, decay, pool)) == 1
    big = torch.zeros(B + 1, Hv, Dk, Dv, device="cuda")
    assert status(lambda: plan.step(*one, decay, big[:-1], state_out=big[1:])) == 1


def test_refusals_without_gpu():
    L = F.lib()
    h = ctypes.c_void_p()
    for dk, dv, dt in ((32, 64, 1), (64, 256, 1), (0, 64, 0), (64, 64, 5)):
        assert L.fftconv_linattn_create(ctypes.byref(h), dk, dv, dt) == 2 and not h.value
    assert L.fftconv_linattn_create(None, 64, 64, 0) == 1
    assert L.fftconv_linattn_destroy(None) == 0
    assert L.fftconv_linattn_scratch_bytes(None, 1, 1, 1, 1, 1, 1) == 0
    a, view = F.LinAttnArgs(), F.View(None, 0, 0, 0)
    assert L.fftconv_linattn_forward(None, ctypes.byref(a), None, view, None, None, 0, None) == 1
    assert L.fftconv_linattn_backward(None, ctypes.byref(a), None, view, None, view, view, view, None, None, 0, None) == 1
    assert L.fftconv_linattn_step(None, ctypes.byref(a), None, None, 0, None, view, None) == 1
    assert L.fftconv_linattn_status(None, None, None) == 1


class Stand:
    """A contiguous CUDA tensor on GPU `index`, as far as the argument checks look."""
    is_cuda = True

    def __init__(self, dtype, shape, index):
        self.dtype, self.shape, self.index = dtype, torch.Size(shape), index

    def get_device(self):
        return self.index

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


@pytest.mark.parametrize("other", ["q", "k", "v", "decay", "offsets"])
def test_tensors_of_another_gpu_are_refused(other, monkeypatch):
    monkeypatch.setattr(F, "_current_device", lambda: 0)
    dt, B, T, H, D = torch.bfloat16, 1, 5, 2, 64
    plan = F.LinearAttention.__new__(F.LinearAttention)  # without a device to create a plan on
    plan.Dk = plan.Dv = D
    plan.torch_dtype, plan._scale, plan._h = dt, 1.0, None
    kinds = dict(q=(dt, (B, T, H, D)), k=(dt, (B, T, H, D)), v=(dt, (B, T, H, D)), decay=(torch.float32, (H,)),
                 offsets=(torch.int32, (3,)))

    def args(dev):
        x = {n: Stand(*s, dev(n)) for n, s in kinds.items()}
        return plan._args(x["q"], x["k"], x["v"], x["decay"], x["offsets"], None)

    assert args(lambda n: 0).nseq == 2
    for dev in (lambda n: 1 if n == other else 0, lambda n: 1):
        with pytest.raises(ValueError, match="GPU"):
            args(dev)
