"""64-bit definitions of the token mixers, on the CPU, and inputs for them."""
import torch


def delta_rule(q, k, v, g, beta, state=None, scale=1.0):
    """Token by token in float64 (differentiable).  q, k: [B, T, Hk, Dk]; v:
    [B, T, Hv, Dv]; g, beta: [B, T, Hv] -> (o, final state)."""
    q, k, v, g, beta = (x.double() for x in (q, k, v, g, beta))
    B, T, Hv = g.shape
    q, k = (x.repeat_interleave(Hv // x.shape[2], 2) for x in (q, k))
    S = torch.zeros(B, Hv, q.shape[3], v.shape[3], dtype=torch.float64) if state is None else state.double()
    outs = []
    for t in range(T):
        S = S * g[:, t].exp()[..., None, None]
        u = beta[:, t, :, None] * (v[:, t] - torch.einsum("bhd,bhde->bhe", k[:, t], S))
        S = S + torch.einsum("bhd,bhe->bhde", k[:, t], u)
        outs.append(scale * torch.einsum("bhd,bhde->bhe", q[:, t], S))
    o = torch.stack(outs, 1) if outs else torch.zeros(B, 0, Hv, v.shape[3], dtype=torch.float64)
    return o, S


def delta_inputs(B, T, Hk, Hv, Dk, Dv, dtype, seed=0):
    """Keys and queries of norm 1, gates as sigmoids and small decays."""
    gen = torch.Generator().manual_seed(seed)

    def n(*s):
        return torch.randn(*s, generator=gen, dtype=torch.float64)

    def unit(x):
        return (x / x.norm(dim=-1, keepdim=True)).to(dtype)

    common = n(B, 1, Hk, Dk)
    q, k = unit(n(B, T, Hk, Dk) + 0.5 * common), unit(n(B, T, Hk, Dk) + 0.5 * common)
    v = n(B, T, Hv, Dv).to(dtype)
    g = (-0.15 * torch.rand(B, T, Hv, generator=gen, dtype=torch.float64)).to(dtype)
    beta = torch.sigmoid(n(B, T, Hv)).to(dtype)
    return q, k, v, g, beta


def qk_norm(x, w, norm, eps, cos=None, sin=None, pos=None, interleaved=False):
    """Norm and rotation of one tensor [B, T, H, D] in float64 (differentiable)."""
    x = x.double()
    m = x.pow(2).mean(-1, keepdim=True) if norm == "rms" else x.pow(2).sum(-1, keepdim=True)
    z = x / (m + eps).sqrt()
    if w is not None:
        z = z * w.double()
    if cos is None or cos.shape[1] == 0:
        return z
    R = 2 * cos.shape[1]
    c, s = cos.double()[pos.long()][:, :, None], sin.double()[pos.long()][:, :, None]
    i = torch.arange(R // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    rot = torch.empty(R, dtype=torch.long)
    rot[a], rot[b] = i, i + R // 2  # where each feature's result sits in the concatenation below
    turned = torch.cat([z[..., a] * c - z[..., b] * s, z[..., b] * c + z[..., a] * s], -1)[..., rot]
    return torch.cat([turned, z[..., R:]], -1)


def rel(got, ref):
    """Distance over size, in the 2-norm; 0 for two zero tensors."""
    got, ref = got.double().cpu(), ref.double()
    d, n = float((got - ref).norm()), float(ref.norm())
    return 0.0 if d == 0 else d / max(n, 1e-300)
