"""Linear attention and layer norm as a model runs them: normed hidden states into the
mixer, its heads normed, the gradients back through all of it, a prompt continued token
by token; and the mixer over rows that are cut into few segments and queues of many
prompts.

Tolerances (2-norm of the difference over that of the result; u = 2^-8 for bf16, 2^-11
for fp16, the largest error of one rounding, 0.43 u its root mean square): o and the
gradients of one call: u, as each is rounded once and has two operands that are (0.75 u).
States: float32 sums, of 12 additions a chunk of 64 tokens and one for each later chunk,
each off by 2^-23 at most.
"""
import pytest
import torch

import fft_long_convolution_gb300 as F
from _attention import attention_chunks, attention_grads, attention_inputs, layer_norm, linear_attention, rel, states

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
DTYPES = [torch.bfloat16, torch.float16]
NAMES = ("dq", "dk", "dv", "dstate")


def test_chunked_definition():
    """The chunked definition is the token-by-token one."""
    ins = attention_inputs(2, 127, 2, 4, 64, 64, torch.bfloat16, seed=1)
    s0 = states(2, 4, 64, 64)
    for got, ref in zip(attention_chunks(*ins, s0, 0.3), linear_attention(*ins, s0, 0.3)):
        assert rel(got, ref) < 1e-12


# 40 chunks of 64 tokens on 152 SMs: 60 rows of heads are cut into two segments, 40 into
# three; of a training step's three walks 24 are cut into two and 14 into three.
@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("B,Hk,Hv,Dk,Dv", [(1, 30, 60, 64, 64), (10, 4, 4, 64, 128), (2, 12, 12, 128, 64), (7, 1, 2, 64, 64),
                                           (2, 7, 7, 128, 128)])
def test_few_segments(B, Hk, Hv, Dk, Dv, dt):
    T = 2550
    ins = [x.cuda() for x in attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=11)]
    do = attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=12)[2].cuda()
    s0, ds = states(B, Hv, Dk, Dv).cuda(), states(B, Hv, Dk, Dv, seed=13).cuda()
    plan = F.LinearAttention(Dk, Dv, dt)
    o, s = plan.forward(*ins, state=s0)
    got = plan.backward(do, *ins, state=s0, dstate=ds)
    again = plan.backward(do, *ins, state=s0, dstate=ds)
    xs = [x.double().requires_grad_() for x in (*ins[:3], s0)]
    ro, rs = attention_chunks(*xs[:3], ins[3], xs[3], Dk ** -0.5)
    assert rel(o, ro.detach()) < U[dt] and rel(s, rs.detach()) < 6.2e-6  # (12 + 40) 2^-23
    ref = torch.autograd.grad((ro * do.double()).sum() + (rs * ds.double()).sum(), xs)
    for name, x, y, z in zip(NAMES, got, ref, again):
        assert rel(x, y) < (6.2e-6 if name == "dstate" else U[dt]), name
        assert torch.equal(x, z), name
    assert plan.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n", [31, 32, 33, 70])
def test_queues_of_many_prompts(n):
    """Up to 32 sequences are taken in the order of their lengths, equal ones among them."""
    dt, Hk, Hv, Dk, Dv = torch.bfloat16, 3, 6, 64, 64
    lens = [(37 * i * i) % 190 if i % 5 else 64 for i in range(n)]
    T = sum(lens) + 3
    ins = attention_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=n)
    do = attention_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=n + 1)[2]
    s0, ds = states(n, Hv, Dk, Dv), states(n, Hv, Dk, Dv, seed=2)
    off = torch.zeros(n + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(torch.tensor(lens), 0)
    plan = F.LinearAttention(Dk, Dv, dt)
    dins = [x.cuda() for x in ins]
    o, s = plan.forward(*dins, state=s0.cuda(), offsets=off.cuda())
    got = plan.backward(do.cuda(), *dins, state=s0.cuda(), dstate=ds.cuda(), offsets=off.cuda())
    for i, L in enumerate(lens):
        at = slice(int(off[i]), int(off[i]) + L)
        part = [x[:, at] for x in ins[:3]] + [ins[3]]
        ref, sref = linear_attention(*part, state=s0[i:i + 1], scale=Dk ** -0.5)
        assert rel(o[:, at], ref) < U[dt] and rel(s[i:i + 1], sref) < 4e-6, i
        if L:
            r = attention_grads(*part, do[:, at], s0[i:i + 1], ds[i:i + 1], Dk ** -0.5)
            for name, x, y in zip(NAMES[:3], got, r):
                assert rel(x[:, at], y) < U[dt], (name, i)
            assert rel(got[3][i:i + 1], r[3]) < 4e-6, i
    assert not any(bool(x[:, T - 3:].any()) for x in (o, *got[:3]))
    assert plan.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 64)])
def test_skewed_queue(Dk, Dv, dt):
    """One prompt as long as all the others: 20 of 90 chunks on average, cut at 360 chunks.
    Up to 938 chunks: (12 + 938) 2^-23 for the states."""
    Hk, Hv = 2, 4
    lens = [1, 0, 60000, 64, 23040, 23041, 5000] + [300] * 12
    lens.append(20 * 90 * 64 - sum(lens))
    n, T = len(lens), sum(lens)
    ins = [x.cuda() for x in attention_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=71)]
    do = attention_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=72)[2].cuda()
    s0, ds = states(n, Hv, Dk, Dv).cuda(), states(n, Hv, Dk, Dv, seed=73).cuda()
    off = torch.zeros(n + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(torch.tensor(lens), 0)
    plan = F.LinearAttention(Dk, Dv, dt)
    o, s = plan.forward(*ins, state=s0, offsets=off.cuda())
    got = plan.backward(do, *ins, state=s0, dstate=ds, offsets=off.cuda())
    for i, L in enumerate(lens):
        if not L:
            assert torch.equal(s[i], s0[i]) and torch.equal(got[3][i], ds[i])
            continue
        at = slice(int(off[i]), int(off[i]) + L)
        xs = [x.double().requires_grad_() for x in (*[y[:, at] for y in ins[:3]], s0[i:i + 1])]
        ro, rs = attention_chunks(*xs[:3], ins[3], xs[3], Dk ** -0.5)
        assert rel(o[:, at], ro.detach()) < U[dt] and rel(s[i:i + 1], rs.detach()) < 1.2e-4, i
        ref = torch.autograd.grad((ro * do[:, at].double()).sum() + (rs * ds[i:i + 1].double()).sum(), xs)
        for name, x, y in zip(NAMES[:3], got, ref):
            assert rel(x[:, at], y) < U[dt], (name, i)
        assert rel(got[3][i:i + 1], ref[3]) < 1.2e-4, i
    assert plan.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [70, 2550])
def test_gradients_of_final_states_without_initial_ones(T):
    dt, B, Hk, Hv, Dk, Dv = torch.bfloat16, 2, 1, 2, 64, 128
    ins = [x.cuda() for x in attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=21)]
    do = attention_inputs(B, T, Hk, Hv, Dk, Dv, dt, seed=22)[2].cuda()
    ds = states(B, Hv, Dk, Dv).cuda()
    plan = F.LinearAttention(Dk, Dv, dt)
    *got, none = plan.backward(do, *ins, dstate=ds)
    xs = [x.double().requires_grad_() for x in ins[:3]]
    o, s = attention_chunks(*xs, ins[3], None, Dk ** -0.5)
    ref = torch.autograd.grad((o * do.double()).sum() + (s * ds.double()).sum(), xs)
    assert none is None and all(rel(x, y) < U[dt] for x, y in zip(got, ref))
    assert plan.device_status() == 0


@pytest.mark.gpu
def test_step_of_no_tokens_passes_states_through():
    dt = torch.bfloat16
    plan = F.LinearAttention(64, 64, dt)
    q, v = torch.empty(2, 0, 1, 64, dtype=dt, device="cuda"), torch.empty(2, 0, 2, 64, dtype=dt, device="cuda")
    decay = torch.zeros(2, device="cuda")
    pool = states(4, 2, 64, 64).cuda()
    kept, out = pool.clone(), torch.full_like(pool, 7.0)
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    assert plan.step(q, q, v, decay, pool, slots=slots).shape == v.shape and torch.equal(pool, kept)
    plan.step(q, q, v, decay, pool, state_out=out, slots=slots)
    assert torch.equal(out[[1, 3]], kept[[1, 3]]) and bool((out[[0, 2]] == 7.0).all()) and torch.equal(pool, kept)


@pytest.mark.gpu
@pytest.mark.parametrize("rate", [0.25, 0.5, 2.0])
def test_fp16_states_of_tokens_long_gone(rate):
    """Tokens with nothing behind them for the rest of their chunk.  A weight is within
    2^-25 of l^i, and the parts within 2^-21 of the product: the error of the state is at
    most (2^-25 + 2^-21 l^i) |k| |v| of each token, doubled for the sums."""
    dt, T, n, D = torch.float16, 64, 24, 64
    q, k, v, _ = attention_inputs(1, T, 1, 1, D, D, dt, seed=31)
    k[:, n:], v[:, n:] = 0, 0
    decay = torch.tensor([-rate])
    _, ref = linear_attention(q, k, v, decay)
    plan = F.LinearAttention(D, D, dt)
    s = plan.forward(q.cuda(), k.cuda(), v.cuda(), decay.cuda())[1].cpu().double()
    w = (-rate * (T - 1 - torch.arange(T, dtype=torch.float64))).exp()
    size = torch.einsum("tk,tv,t->kv", k[0, :, 0].double().abs(), v[0, :, 0].double().abs(), 2.0 ** -25 + 2.0 ** -21 * w)
    assert bool(((s - ref)[0, 0].abs() <= 2 * size).all())


class Block:
    """x + heads normed (attention (projections of normed x)), with all its gradients."""

    def __init__(self, D, Hk, Hv, d, dt, seed=5):
        gen = torch.Generator().manual_seed(seed)

        def n(*s):
            return torch.randn(*s, generator=gen)

        self.D, self.Hk, self.Hv, self.d, self.dt = D, Hk, Hv, d, dt
        self.w, self.b = (1.0 + 0.1 * n(D)).cuda(), (0.1 * n(D)).cuda()
        self.wh, self.bh = (1.0 + 0.1 * n(Hv, d)).cuda(), (0.1 * n(Hv, d)).cuda()
        self.proj = (n(D, (2 * Hk + Hv) * d) / D ** 0.5).to(dt).cuda()
        self.decay = torch.log1p(-torch.exp2(-(3.0 + 5.0 * torch.rand(Hv, generator=gen)))).cuda()
        self.norm, self.heads = F.LayerNorm(D, dt), F.LayerNorm(d, dt)
        self.mix = F.LinearAttention(d, d, dt)

    def split(self, y):
        B, T, _ = y.shape
        q, k, v = y.split([self.Hk * self.d, self.Hk * self.d, self.Hv * self.d], -1)
        return q.view(B, T, self.Hk, self.d), k.view(B, T, self.Hk, self.d), v.view(B, T, self.Hv, self.d)

    def forward(self, x, state=None):
        n = self.norm.forward(x, self.w, self.b)
        qkv = n @ self.proj
        o, s = self.mix.forward(*self.split(qkv), self.decay, state=state)
        return self.heads.forward(o, self.wh, self.bh), s, (x, n, qkv, o, state)

    def backward(self, dy, saved, ds):
        x, n, qkv, o, state = saved
        do, dwh, dbh = self.heads.backward(dy, o, self.wh, self.bh)
        dq, dk, dv, d0 = self.mix.backward(do, *self.split(qkv), self.decay, state=state, dstate=ds)
        dqkv = torch.cat([g.flatten(2) for g in (dq, dk, dv)], -1)
        dx, dw, db = self.norm.backward(dqkv @ self.proj.T, x, self.w, self.b)
        return dict(dx=dx, dw=dw, db=db, dwh=dwh, dbh=dbh, dstate=d0, dproj=n.flatten(0, 1).T @ dqkv.flatten(0, 1))

    def exact(self, x, state):
        """In float64, differentiable: (outputs, final state), and the leaves."""
        leaves = dict(dx=x, dw=self.w, db=self.b, dwh=self.wh, dbh=self.bh, dstate=state, dproj=self.proj)
        leaves = {k: t.detach().double().requires_grad_() for k, t in leaves.items()}
        n = layer_norm(leaves["dx"], leaves["dw"], leaves["db"])
        o, s = attention_chunks(*self.split(n @ leaves["dproj"]), self.decay, leaves["dstate"], self.d ** -0.5)
        return layer_norm(o, leaves["dwh"], leaves["dbh"]), s, leaves


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("D,Hk,Hv,d,B,T", [(768, 6, 6, 128, 2, 131), (768, 6, 12, 64, 3, 77), (256, 1, 2, 64, 1, 1)])
def test_training_step_of_a_block(D, Hk, Hv, d, B, T, dt):
    """Forward: the norm's output, its projections (0.43 u each, and what they inherit) and o
    (0.75 u) make sqrt(3) 0.61 u + 0.75 u at most, which the heads' norm passes on at a
    rate of |o| / std(o) < 1.5, and rounds: 3 u.  Gradients: three more roundings of that
    kind on the way back (do, dqkv, dn), on operands that are off by the above: twice it,
    6 u; states and their gradients, of 16-bit operands: 3 u and 6 u."""
    block = Block(D, Hk, Hv, d, dt)
    gen = torch.Generator().manual_seed(7)
    x = torch.randn(B, T, D, generator=gen).to(dt).cuda()
    dy = torch.randn(B, T, Hv, d, generator=gen).to(dt).cuda()
    s0, ds = states(B, Hv, d, d).cuda(), states(B, Hv, d, d, seed=3).cuda()
    y, s, saved = block.forward(x, s0)
    grads = block.backward(dy, saved, ds)
    ry, rs, leaves = block.exact(x, s0)
    assert rel(y, ry.detach()) < 3 * U[dt] and rel(s, rs.detach()) < 3 * U[dt]
    ref = torch.autograd.grad((ry * dy.double()).sum() + (rs * ds.double()).sum(), list(leaves.values()))
    for name, r in zip(leaves, ref):
        assert rel(grads[name], r) < 6 * U[dt], name
    assert block.mix.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
def test_prompt_then_decoding(dt):
    """A prompt's states go on into single tokens, each normed before and after."""
    block = Block(768, 6, 12, 64, dt)
    B, T, n = 3, 90, 6
    x = torch.randn(B, T, 768, generator=torch.Generator().manual_seed(8)).to(dt).cuda()
    y, s, _ = block.forward(x[:, :T - n])
    pool = torch.zeros(7, 12, 64, 64, device="cuda")
    slots = torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")
    pool[slots.long()] = s
    out = [y]
    for t in range(T - n, T):
        q = block.split(block.norm.forward(x[:, t:t + 1], block.w, block.b) @ block.proj)
        o = block.mix.step(*q, block.decay, pool, slots=slots)
        out.append(block.heads.forward(o, block.wh, block.bh))
    ry, rs = (t.detach() for t in block.exact(x, torch.zeros_like(s))[:2])
    y = torch.cat(out, 1)
    assert rel(y[:, :T - n], ry[:, :T - n]) < 3 * U[dt] and rel(y[:, T - n:], ry[:, T - n:]) < 3 * U[dt]
    assert rel(pool[slots.long()], rs) < 3 * U[dt] and not bool(pool[[1, 2, 4, 6]].any())
    whole, s, _ = block.forward(x)
    assert rel(y, whole) < 3 * U[dt] and rel(pool[slots.long()], s) < 3 * U[dt]


class Stand:
    """A contiguous tensor of one GPU, as far as a call looks before it is refused."""

    def __init__(self, dtype, shape, dev):
        self.dtype, self.shape, self.dev = dtype, torch.Size(shape), dev
        self.is_cuda = True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.dev

    def data_ptr(self):
        return 1 << 20


@pytest.mark.parametrize("other", ["x", "w", "b"])
def test_norm_with_tensors_of_another_gpu_is_refused(other, monkeypatch):
    monkeypatch.setattr(F, "_current_device", lambda: 0)
    norm = F.LayerNorm(64, torch.bfloat16)
    kinds = dict(x=(torch.bfloat16, (2, 5, 64)), w=(torch.float32, (64,)), b=(torch.float32, (64,)))

    def args(dev):
        return norm._args(*[Stand(*s, dev(n)) for n, s in kinds.items()])

    assert args(lambda n: 0).T == 5
    for dev in (lambda n: 1 if n == other else 0, lambda n: 1):
        with pytest.raises(ValueError, match="GPU"):
            args(dev)
    x = Stand(*kinds["x"], 0)
    for what in ("y", "dy", "dx"):
        with pytest.raises(ValueError, match="GPU"):
            norm._view(Stand(*kinds["x"], 1), what, x.shape, 0)
