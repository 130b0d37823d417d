"""64-bit definitions of the linear attention and the layer norm, on the CPU, and inputs for them."""
import torch

LOWEST = -1e4  # a log decay whose exponential is zero in 64 bits


def linear_attention(q, k, v, decay, state=None, scale=1.0):
    """Token by token in float64 (differentiable).  q, k: [B, T, Hk, Dk]; v:
    [B, T, Hv, Dv]; decay: [Hv] logarithms -> (o, final state)."""
    q, k, v = (x.double() for x in (q, k, v))
    B, T, Hv, Dv = v.shape
    lam = decay.double().clamp(LOWEST, 0.0).exp()[None, :, None, None]
    q, k = (x.repeat_interleave(Hv // x.shape[2], 2) for x in (q, k))
    S = torch.zeros(B, Hv, q.shape[3], Dv, dtype=torch.float64) if state is None else state.double()
    outs = []
    for t in range(T):
        S = lam * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        outs.append(scale * (q[:, t, :, :, None] * S).sum(-2))
    return torch.stack(outs, 1) if outs else torch.zeros(B, 0, Hv, Dv, dtype=torch.float64), S


def attention_inputs(B, T, Hk, Hv, Dk, Dv, dtype, seed=0):
    """Queries and keys with something in common, decays from 1 - 2^-3 to 1 - 2^-12."""
    gen = torch.Generator().manual_seed(seed)

    def n(*s):
        return torch.randn(*s, generator=gen, dtype=torch.float64)

    q, k = ((0.9 * n(B, T, Hk, Dk) + 0.4 * n(B, 1, Hk, Dk)).to(dtype) for _ in range(2))
    decay = torch.log1p(-torch.exp2(-(3.0 + 9.0 * torch.rand(Hv, generator=gen, dtype=torch.float64)))).float()
    return q, k, n(B, T, Hv, Dv).to(dtype), decay


def states(n, Hv, Dk, Dv, seed=9):
    return torch.randn(n, Hv, Dk, Dv, generator=torch.Generator().manual_seed(seed))


def attention_grads(q, k, v, decay, do, s0, ds, scale):
    """(dq, dk, dv, gradient of the initial state) of <o, do> + <final state, ds>, by the chain rule."""
    xs = [x.double().requires_grad_() for x in (q, k, v)] + [s0.double().requires_grad_()]
    o, s = linear_attention(*xs[:3], decay, xs[3], scale)
    return torch.autograd.grad((o * do.double()).sum() + (s * ds.double()).sum(), xs)


def layer_norm(x, w=None, b=None, eps=1e-5):
    """In float64 (differentiable)."""
    x = x.double()
    c = x - x.mean(-1, keepdim=True)
    y = c / (c.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    y = y if w is None else y * w.double()
    return y if b is None else y + b.double()


def rel(got, ref):
    """Distance over size, in the 2-norm; 0 for two zero tensors."""
    got, ref = got.double().cpu(), ref.double().cpu()
    d, n = float((got - ref).norm()), float(ref.norm())
    return 0.0 if d == 0 else d / max(n, 1e-300)


def attention_chunks(q, k, v, decay, state=None, scale=1.0, C=50):
    """linear_attention by chunks of C tokens, on the inputs' device, for rows too long to
    take token by token."""
    q, k, v = (x.double() for x in (q, k, v))
    B, T, Hv, Dv = v.shape
    g = decay.double().clamp(LOWEST, 0.0)
    q, k = (x.repeat_interleave(Hv // x.shape[2], 2) for x in (q, k))
    S = torch.zeros(B, Hv, q.shape[3], Dv, dtype=torch.float64, device=v.device) if state is None else state.double()
    outs = []
    for t in range(0, T, C):
        x, y, z = (a[:, t:t + C] for a in (q, k, v))
        m = x.shape[1]
        i = torch.arange(m, device=v.device, dtype=torch.float64)
        D = torch.where(i[:, None] >= i, (g[:, None, None] * (i[:, None] - i)).exp(), 0.0)
        P = torch.einsum("bihd,bjhd->bhij", x, y) * D
        o = torch.einsum("bihd,bhde->bihe", x * (g * (i[:, None] + 1)).exp()[..., None], S)
        outs.append(scale * (o + torch.einsum("bhij,bjhe->bihe", P, z)))
        S = (g * m).exp()[:, None, None] * S + torch.einsum("bjhd,bjhe->bhde", y * (g * (m - 1 - i)[:, None]).exp()[..., None], z)
    return torch.cat(outs, 1), S
