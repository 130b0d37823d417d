"""Cases of linear attention with a decay for each head and of the layer norm.

Every case is one pass of an operator: a prompt through the attention (outputs
and final states), a training step of it (outputs, final states and gradients),
a decoding step (outputs and updated states), the norm of rows of features,
forward or as a training step.  With ``own`` false the pass is computed in
elementary float32 operations.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_CHUNK = 256


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one prompt of 262144 tokens (the longest row of the 512 x 512 image workload), hidden 768 as 6 heads of 128
        dict(name="prefill-256k", op="prefill", B=1, T=262144, Hk=6, Hv=6, Dk=128, Dv=128, dtype="bf16", ragged=0, init=False),
        # a batch of 4096-token prompts at hidden 768, continuing from given states
        dict(name="prefill-4k", op="prefill", B=8, T=4096, Hk=6, Hv=6, Dk=128, Dv=128, dtype="bf16", ragged=0, init=True),
        # 24 prompts of uneven length packed into one row (a serving queue), fp16, two value heads to a key head
        dict(name="prefill-ragged", op="prefill", B=1, T=16411, Hk=6, Hv=12, Dk=64, Dv=128, dtype="fp16", ragged=24, init=True),
        # a training step on 4096-token rows at hidden 768
        dict(name="train-4k", op="train", B=8, T=4096, Hk=6, Hv=6, Dk=128, Dv=128, dtype="bf16", ragged=0, init=False),
        # a training step on rows of 1000 samples that continue earlier ones, 12 heads of 64, shared keys, fp16
        dict(name="train-1k", op="train", B=16, T=1000, Hk=6, Hv=12, Dk=64, Dv=64, dtype="fp16", ragged=0, init=True),
        # one user decoding: latency
        dict(name="step-1", op="step", B=1, T=1, Hk=6, Hv=6, Dk=128, Dv=128, dtype="bf16", slots=False),
        # a full serving batch, one token for each of 256 users, their states scattered over a pool
        dict(name="step-256", op="step", B=256, T=1, Hk=6, Hv=12, Dk=128, Dv=128, dtype="bf16", slots=True),
        # norm of one token for each of 8 users, hidden 768
        dict(name="norm-8x1", op="norm", B=8, T=1, H=1, D=768, dtype="bf16", affine=True, train=False),
        # norm of gene-length rows: two million positions of 32 features
        dict(name="norm-2m", op="norm", B=1, T=2097152, H=1, D=32, dtype="bf16", affine=True, train=False),
        # a training step of the norm at the longest row of the 16K workload, hidden 768
        dict(name="norm-train-16k", op="norm", B=8, T=16384, H=1, D=768, dtype="bf16", affine=True, train=True),
        # the mixer's outputs normed for each head, a training step on odd sizes, fp16
        dict(name="norm-train-heads", op="norm", B=5, T=1023, H=12, D=64, dtype="fp16", affine=True, train=True),
        # a wide row, a training step without weights
        dict(name="norm-train-wide", op="norm", B=3, T=501, H=1, D=5000, dtype="bf16", affine=False, train=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "train", "train", "step", "step", "norm", "norm", "norm"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "norm":
        if rng.random() < 0.4:
            H, D = rng.randint(2, 16), rng.choice([32, 64, 64, 80, 128, 128, 256])
        else:
            H, D = 1, 8 * _log_int(rng, 1, 1024)
        tokens = _log_int(rng, 1, min(2 ** 21, 2 ** 26 // (H * D)))
        B = min(tokens, _log_int(rng, 1, 64))
        return dict(op=op, B=B, T=max(1, tokens // B), H=H, D=D, dtype=dtype, affine=rng.random() < 0.8, train=rng.random() < 0.5)
    Dk, Dv = rng.choice([64, 128]), rng.choice([64, 128])
    if op == "step":
        Hk = rng.randint(1, 12)
        return dict(op=op, B=_log_int(rng, 1, 256), T=rng.choice([1, 1, 1, 2, 5]), Hk=Hk, Hv=Hk * rng.choice([1, 1, 2]), Dk=Dk,
                    Dv=Dv, dtype=dtype, slots=rng.random() < 0.5)
    Hk = rng.randint(1, 6)
    Hv = Hk * rng.choice([1, 1, 2])
    tokens = _log_int(rng, 16, min(32768 if op == "train" else 65536, 32768 * 12 // Hv))
    if rng.random() < 0.4:
        B, T, ragged = 1, tokens, rng.randint(1, min(tokens, 32))
    else:
        B = min(tokens, _log_int(rng, 1, 32))
        T, ragged = max(1, tokens // B), 0
    return dict(op=op, B=B, T=T, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, dtype=dtype, ragged=ragged, init=rng.random() < 0.5)


# ------------------------------------------------------------------- inputs

def _lengths(n, total, seed):
    """n uneven lengths that sum to total; one of them 0 where there is room."""
    if n == 1:
        return [total]
    gen = torch.Generator().manual_seed(seed)
    w = torch.rand(n, generator=gen, dtype=torch.float64) ** 2 + 1e-3
    if n > 3:
        w[n // 2] = 0.0
    cut = torch.floor(torch.cumsum(w, 0) / w.sum() * total + 0.5).long()
    cut[-1] = total
    return torch.diff(cut, prepend=torch.zeros(1, dtype=torch.long)).tolist()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = _DT[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    st = {"case": case, "dt": dt}
    B, T = case["B"], case["T"]
    if case["op"] == "norm":
        H, D = case["H"], case["D"]
        shape, ws = ((B, T, D), (D,)) if H == 1 else ((B, T, H, D), (H, D))
        # a residual stream: features of unlike size with a mean of their own
        st["x"] = (normal(*shape) * (0.5 + torch.rand(*ws, generator=gen, device=dev)) + 0.3 * normal(*ws)).to(dt)
        st["w"] = st["b"] = None
        if case["affine"]:
            st["w"], st["b"] = 1.0 + 0.2 * normal(*ws), 0.1 * normal(*ws)
        if case["train"]:
            st["dy"] = normal(*shape).to(dt)
        st["eps"] = 1e-5
        if own:
            import fft_long_convolution_gb300 as F
            st["plan"] = F.LayerNorm(D, dt, eps=st["eps"])
        return st

    Hk, Hv, Dk, Dv = case["Hk"], case["Hv"], case["Dk"], case["Dv"]

    def keys(*shape):  # rows of one sequence have something in common
        return (0.9 * normal(*shape) + 0.45 * normal(shape[0], 1, *shape[2:])).to(dt)

    st["q"], st["k"] = keys(B, T, Hk, Dk), keys(B, T, Hk, Dk)
    st["v"] = normal(B, T, Hv, Dv).to(dt)
    # decays of the heads from 1 - 2^-5 to 1 - 2^-12, as logarithms
    at = 5.0 + 7.0 * (torch.arange(Hv, device=dev, dtype=torch.float64) + torch.rand((), generator=gen, device=dev).double()) / Hv
    st["decay"] = torch.log1p(-torch.exp2(-at)).float()
    st["scale"] = Dk ** -0.5
    if case["op"] == "step":
        n, st["slots"] = B, None
        if case["slots"]:
            n = B + B // 2 + 1
            st["slots"] = torch.randperm(n, generator=gen, device=dev)[:B].to(torch.int32).contiguous()
        st["state"] = normal(n, Hv, Dk, Dv)
        st["next"] = st["state"].clone()  # the pool that receives the updated states
    else:
        st["offsets"], st["lens"], n = None, [T] * B, B
        if case["ragged"]:
            n = case["ragged"]
            st["lens"] = _lengths(n, T, seed)
            off = torch.zeros(n + 1, dtype=torch.long)
            off[1:] = torch.cumsum(torch.tensor(st["lens"]), 0)
            st["offsets"] = off.to(torch.int32).to(dev)
        st["state"] = normal(n, Hv, Dk, Dv) if case["init"] else None
        if case["op"] == "train":
            st["do"] = normal(B, T, Hv, Dv).to(dt)
            # rows that continue earlier ones are continued themselves
            st["dstate"] = normal(n, Hv, Dk, Dv) if case["init"] else None
    if own:
        import fft_long_convolution_gb300 as F
        st["plan"] = F.LinearAttention(Dk, Dv, dt)
    return st


# ------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if op == "norm":
        return _norm_own(state) if own else _norm_plain(state)
    if op == "step":
        return _step_own(state) if own else _step_plain(state)
    return _attention_own(state) if own else _attention_plain(state)


def _norm_own(s):
    y = s["plan"].forward(s["x"], s["w"], s["b"])
    if not s["case"]["train"]:
        return {"y": y}
    dx, dw, db = s["plan"].backward(s["dy"], s["x"], s["w"], s["b"])
    return {"y": y, "dx": dx, "dw": dw, "db": db}


def _step_own(s):
    o = s["plan"].step(s["q"], s["k"], s["v"], s["decay"], s["state"], state_out=s["next"], slots=s["slots"], scale=s["scale"])
    return {"o": o, "state": s["next"]}


def _attention_own(s):
    p, args = s["plan"], (s["q"], s["k"], s["v"], s["decay"])
    kw = dict(state=s["state"], offsets=s["offsets"], scale=s["scale"])
    o, state = p.forward(*args, **kw)
    out = {"o": o, "state": state}
    if s["case"]["op"] == "train":
        out["dq"], out["dk"], out["dv"], dstate = p.backward(s["do"], *args, dstate=s["dstate"], **kw)
        if s["state"] is not None:
            out["dstate"] = dstate
    return out


# ------------------------------------------------------------------- plain forms

def _norm_plain(s):
    case, x = s["case"], s["x"].float()
    D = case["D"]
    c = x - x.sum(-1, keepdim=True) / D
    r = torch.rsqrt((c * c).sum(-1, keepdim=True) / D + s["eps"])
    h = c * r
    y = h if s["w"] is None else h * s["w"] + s["b"]
    out = {"y": y.to(s["dt"])}
    if not case["train"]:
        return out
    dy = s["dy"].float()
    dz = dy if s["w"] is None else dy * s["w"]
    dx = r * (dz - dz.sum(-1, keepdim=True) / D - h * ((dz * h).sum(-1, keepdim=True) / D))
    out["dx"] = dx.to(s["dt"])
    out["dw"] = out["db"] = None
    if s["w"] is not None:
        # sums over up to millions of tokens in 64 bits
        out["dw"] = (dy * h).sum((0, 1), dtype=torch.float64).float()
        out["db"] = dy.sum((0, 1), dtype=torch.float64).float()
    return out


def _heads(x, Hv):
    return x.repeat_interleave(Hv // x.shape[2], dim=2) if x.shape[2] != Hv else x


def _step_plain(s):
    case = s["case"]
    Hv = case["Hv"]
    q, k, v = _heads(s["q"], Hv).float(), _heads(s["k"], Hv).float(), s["v"].float()
    lam = s["decay"].exp()[None, :, None, None]
    at = slice(None) if s["slots"] is None else s["slots"].long()
    S = s["state"][at]
    outs = []
    for t in range(case["T"]):
        S = lam * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        outs.append(s["scale"] * (q[:, t, :, :, None] * S).sum(-2))
    s["next"][at] = S
    return {"o": torch.stack(outs, 1).to(s["dt"]), "state": s["next"]}


def _rows(s):
    """The case's sequences as rows of one length, a whole number of chunks, with the gap in front of the first token."""
    dev = s["q"].device
    lens = torch.tensor(s["lens"], device=dev)
    n, top = len(s["lens"]), max(max(s["lens"]), 1)
    C = min(_CHUNK, top)
    top = (top + C - 1) // C * C
    row = torch.repeat_interleave(torch.arange(n, device=dev), lens, output_size=sum(s["lens"]))
    start = torch.cumsum(lens, 0) - lens
    col = torch.arange(sum(s["lens"]), device=dev) - start[row] + (top - lens)[row]

    def put(x):
        """[sequence, head, token, feature], zeros before a sequence's first token."""
        out = torch.zeros(n, top, *x.shape[2:], device=dev, dtype=torch.float32)
        out[row, col] = x.reshape(-1, *x.shape[2:]).float()
        return out.movedim(2, 1)

    def take(x, like):
        x = x.movedim(1, 2)
        return x[row, col].reshape(*like.shape[:2], *x.shape[2:])

    return put, take, C, lens


def _mix(q, k, v, g, C, init=None, at=None):
    """scale-free outputs sum_(j <= i) l^(i-j) (q_i.k_j) v_j, plus l^(i+1) of the initial state `at` tokens in, and
    sum_j l^(T-1-j) k_j v_j^T; whole chunks, every power of the decay from 64 bits."""
    n, H, T, _ = q.shape
    nc = T // C
    q, k, v = (x.reshape(n, H, nc, C, x.shape[3]) for x in (q, k, v))
    i = torch.arange(max(C, nc), device=q.device, dtype=torch.float64)
    g = g.double()[:, None]

    def below(m, step, gap):
        """l^(step (a - b - gap)) for a - b >= gap, [H, m, m]"""
        d = i[:m, None] - i[None, :m] - gap
        return torch.where(d >= 0, (g[:, :, None] * step * d.clamp(min=0)).exp(), 0.0).float()

    o = ((q @ k.transpose(-1, -2)) * below(C, 1, 0)[None, :, None]) @ v
    tail = (g * (C - 1 - i[:C])).exp().float()
    KV = (k * tail[None, :, None, :, None]).transpose(-1, -2) @ v
    flat = KV.flatten(-2)
    S = (below(nc, C, 1)[None] @ flat).reshape(KV.shape)
    last = ((g * C * (nc - 1 - i[:nc])).exp().float()[None, :, None, :] @ flat).reshape(n, H, *KV.shape[-2:])
    o = o + (g * (i[:C] + 1)).exp().float()[None, :, None, :, None] * (q @ S)
    o = o.reshape(n, H, T, v.shape[-1])
    if init is not None:
        t = torch.arange(T, device=q.device, dtype=torch.float64)
        d = t[None, None, :] - at.double()[:, None, None] + 1.0
        w = torch.where(d > 0, (g[None] * d.clamp(min=0)).exp(), 0.0).float()
        o = o + w[..., None] * (q.reshape(n, H, T, -1) @ init)
        last = last + (g[None] * (T - at).double()[:, None, None]).exp().float()[..., None] * init
    return o, last


def _attention_plain(s):
    case, dt, scale = s["case"], s["dt"], s["scale"]
    Hv = case["Hv"]
    put, take, C, lens = _rows(s)
    q, k, v = put(_heads(s["q"], Hv)), put(_heads(s["k"], Hv)), put(s["v"])
    gap = q.shape[2] - lens
    o, last = _mix(q, k, v, s["decay"], C, s["state"], gap)
    out = {"o": (scale * take(o, s["v"])).to(dt), "state": last}
    if case["op"] == "prefill":
        return out
    do = put(s["do"])
    turned = None if s["state"] is None else s["state"].transpose(-1, -2)
    dq = scale * _mix(do, v, k, s["decay"], C, turned, gap)[0]
    # backwards in time: what comes after a token, the gap behind the last one
    rq, rk, rv, rdo = (x.flip(2) for x in (q, k, v, do))
    dv = scale * _mix(rk, rq, rdo, s["decay"], C)[0].flip(2)
    dk = scale * _mix(rv, rdo, rq, s["decay"], C)[0].flip(2)
    T = q.shape[2]
    g = s["decay"].double()[None, :, None]
    if s["dstate"] is not None:
        t = torch.arange(T, device=q.device, dtype=torch.float64)[None, None, :]
        w = (g * (T - 1 - t)).exp().float()[..., None]
        dv, dk = dv + w * (k @ s["dstate"]), dk + w * (v @ s["dstate"].transpose(-1, -2))

    def shared(x):
        return take(x.unflatten(1, (case["Hk"], Hv // case["Hk"])).sum(2), s["q"]).to(dt)

    out.update({"dq": shared(dq), "dk": shared(dk), "dv": take(dv, s["v"]).to(dt)})
    if s["state"] is not None:
        t = torch.arange(T, device=q.device, dtype=torch.float64)
        d = t[None, None, :] - gap.double()[:, None, None] + 1.0
        w = torch.where(d > 0, (g * d.clamp(min=0)).exp(), 0.0).float()
        dS = scale * ((q * w[..., None]).transpose(-1, -2) @ do)
        out["dstate"] = dS + (g * lens.double()[:, None, None]).exp().float()[..., None] * s["dstate"]
    return out


# ------------------------------------------------------------------- the floor

def work(case):
    B, T = case["B"], case["T"]
    if case["op"] == "norm":
        n = B * T * case["H"] * case["D"]
        if not case["train"]:
            return {"bytes": 4 * n, "flops": 7 * n}
        return {"bytes": 10 * n, "flops": 20 * n}
    Hk, Hv, Dk, Dv = case["Hk"], case["Hv"], case["Dk"], case["Dv"]
    qk, vo = 2 * B * T * Hk * Dk * 2, 2 * B * T * Hv * Dv * 2
    flops = 4 * B * T * Hv * Dk * Dv
    if case["op"] == "step":
        return {"bytes": qk + vo + 2 * 4 * B * Hv * Dk * Dv, "flops": flops}
    states = 4 * (case["ragged"] or B) * Hv * Dk * Dv
    if case["op"] == "prefill":
        return {"bytes": qk + vo + states * (2 if case["init"] else 1), "flops": flops}
    # o written, do read, three gradients written; the states and their gradients
    return {"bytes": 2 * qk + 2 * vo + states * (4 if case["init"] else 1), "flops": 3 * flops}


# ------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _norm_exact(s) if case["op"] == "norm" else _attention_exact(s)


def _norm_exact(s):
    x = s["x"].double()
    std, mean = torch.std_mean(x, dim=-1, keepdim=True, correction=0)
    size = (std.square() + s["eps"]).sqrt()
    hat = (x - mean) / size
    w = torch.ones((), device=x.device, dtype=torch.float64) if s["w"] is None else s["w"].double()
    b = 0.0 if s["b"] is None else s["b"].double()
    out = {"y": hat * w + b}
    if s["case"]["train"]:
        dy = s["dy"].double()
        dh = dy * w
        out["dx"] = (dh - dh.mean(-1, keepdim=True) - hat * (dh * hat).mean(-1, keepdim=True)) / size
        out["dw"] = out["db"] = None
        if s["w"] is not None:
            out["dw"], out["db"] = (dy * hat).sum((0, 1)), dy.sum((0, 1))
    return out


def _attention_exact(s):
    """Token by token, all sequences of the case side by side."""
    case = s["case"]
    Hk, Hv, Dk, Dv = case["Hk"], case["Hv"], case["Dk"], case["Dv"]
    train, step = case["op"] == "train", case["op"] == "step"
    lens = [case["T"]] * case["B"] if step else s["lens"]
    n, top = len(lens), max(lens + [1])
    if top * (110e-6 + 6 * n * Hv * Dk * Dv * 8 / 4e12) * (2.5 if train else 1) > 18:
        return None
    dev = s["q"].device
    flat = {m: s[m].double().reshape(-1, *s[m].shape[2:]) for m in ("q", "k", "v") + (("do",) if train else ())}
    total = flat["v"].shape[0]
    size = torch.tensor(lens, device=dev)
    begin = torch.cumsum(size, 0) - size
    group = Hv // Hk
    for m in ("q", "k"):
        flat[m] = flat[m].repeat_interleave(group, 1)
    lam = s["decay"].double().exp()[None, :, None, None]
    if step:
        at = torch.arange(n, device=dev) if s["slots"] is None else s["slots"].long()
        pool = s["state"].double()
        S = pool[at]
    else:
        S = torch.zeros(n, Hv, Dk, Dv, device=dev, dtype=torch.float64) if s["state"] is None else s["state"].double()
    # token t of every sequence, a spare token past the last one for sequences that are over
    times = torch.arange(top, device=dev)
    index = torch.where(times[:, None] < size[None], begin[None] + times[:, None], total)
    even = len(set(lens)) == 1
    live = (times[:, None] < size[None]).double()[..., None, None, None]
    for m in flat:
        flat[m] = torch.cat([flat[m], torch.zeros_like(flat[m][:1])])
    o, dq = (torch.zeros(total + 1, Hv, d, device=dev, dtype=torch.float64) for d in (Dv, Dk))
    dk, dv = torch.zeros_like(dq), torch.zeros_like(o)
    for t in range(top):
        tok = index[t]
        new = torch.addcmul(lam * S, flat["k"][tok].unsqueeze(-1), flat["v"][tok].unsqueeze(-2))
        S = new if even else torch.where(live[t] > 0, new, S)
        o[tok] = s["scale"] * (flat["q"][tok].unsqueeze(-2) @ S).squeeze(-2)
        if train:
            dq[tok] = s["scale"] * (S @ flat["do"][tok].unsqueeze(-1)).squeeze(-1)
    shape = s["v"].shape
    if step:
        pool[at] = S
        return {"o": o[:total].reshape(shape), "state": pool}
    out = {"o": o[:total].reshape(shape), "state": S}
    if not train:
        return out
    R = torch.zeros_like(S) if s["dstate"] is None else s["dstate"].double()
    for t in range(top - 1, -1, -1):
        tok = index[t]
        new = torch.addcmul(R, flat["q"][tok].unsqueeze(-1) * s["scale"], flat["do"][tok].unsqueeze(-2))
        dv[tok] = (flat["k"][tok].unsqueeze(-2) @ new).squeeze(-2)
        dk[tok] = (new @ flat["v"][tok].unsqueeze(-1)).squeeze(-1)
        R = lam * new if even else torch.where(live[t] > 0, lam * new, R)
    ks = s["k"].shape
    out["dq"], out["dk"] = (x[:total].reshape(*ks[:2], Hk, group, Dk).sum(3) for x in (dq, dk))
    out["dv"] = dv[:total].reshape(shape)
    if s["state"] is not None:
        out["dstate"] = R
    return out
