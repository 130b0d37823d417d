"""Cases of the gated delta rule and of the query/key norm with rotation.

Every case is one pass of an operator: a prompt through the chunked delta rule
(outputs and final states), a training step of it (outputs and gradients), a
decoding step (outputs and updated states), the norm and rotation of queries
and keys, forward or as a training step.  With ``own`` false the pass is
computed in elementary float32 operations.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_CHUNK = 64


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one prompt of 262144 tokens (the longest row of the 512 x 512 image workload), hidden 768 as 6 heads of 128
        dict(name="prefill-256k", op="prefill", B=1, T=262144, Hk=6, Hv=6, Dk=128, Dv=128, dtype="bf16", ragged=0, init=False),
        # a batch of 4096-token prompts at hidden 768, 6 heads of 128, continuing from given states
        dict(name="prefill-4k", op="prefill", B=8, T=4096, Hk=6, Hv=6, Dk=128, Dv=128, dtype="bf16", ragged=0, init=True),
        # 24 prompts of uneven length packed into one row (a serving queue), fp16, two value heads to a key head
        dict(name="prefill-ragged", op="prefill", B=1, T=16411, Hk=6, Hv=12, Dk=64, Dv=128, dtype="fp16", ragged=24, init=True),
        # a training step on 4096-token rows at hidden 768
        dict(name="train-4k", op="train", B=8, T=4096, Hk=6, Hv=6, Dk=128, Dv=128, dtype="bf16", ragged=0, init=False),
        # a training step on rows of 1000 samples (not a whole number of chunks), 12 heads of 64, shared keys, fp16
        dict(name="train-1k", op="train", B=16, T=1000, Hk=6, Hv=12, Dk=64, Dv=64, dtype="fp16", ragged=0, init=False),
        # one user decoding: latency
        dict(name="step-1", op="step", B=1, T=1, Hk=6, Hv=6, Dk=128, Dv=128, dtype="bf16", slots=False),
        # a full serving batch, one token for each of 256 users, their states scattered over a pool
        dict(name="step-256", op="step", B=256, T=1, Hk=6, Hv=12, Dk=128, Dv=128, dtype="bf16", slots=True),
        # four tokens at once for each of 33 users (a draft accepted as a whole), fp16
        dict(name="step-33x4", op="step", B=33, T=4, Hk=12, Hv=12, Dk=64, Dv=64, dtype="fp16", slots=True),
        # norm and rotation of one token for each of 8 users
        dict(name="norm-8x1", op="norm", B=8, T=1, Hq=6, Hk=6, D=128, R=128, kind="rms", inter=False, dtype="bf16", train=False),
        # norm and rotation of a batch of prompts
        dict(name="norm-8x4k", op="norm", B=8, T=4096, Hq=12, Hk=6, D=64, R=32, kind="l2", inter=True, dtype="bf16", train=False),
        # the same in a training step at the longest row of the 16K workload
        dict(name="norm-train-16k", op="norm", B=8, T=16384, Hq=6, Hk=6, D=128, R=128, kind="rms", inter=False, dtype="bf16", train=True),
        # a training step with odd sizes: 80 features, half of them rotated, fewer key heads
        dict(name="norm-train-odd", op="norm", B=5, T=1023, Hq=9, Hk=3, D=80, R=40, kind="rms", inter=False, dtype="fp16", train=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "train", "train", "step", "step", "norm", "norm"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "norm":
        D = rng.choice([64, 64, 80, 96, 128, 128, 256])
        R = rng.choice([0, D // 2, D])
        Hk = rng.randint(1, 8)
        Hq = Hk * rng.choice([1, 2, 3])
        tokens = _log_int(rng, 1, min(131072, 3 * 2 ** 25 // ((Hq + Hk) * D)))
        B = min(tokens, _log_int(rng, 1, 64))
        return dict(op=op, B=B, T=max(1, tokens // B), Hq=Hq, Hk=Hk, D=D, R=R, kind=rng.choice(["rms", "l2"]),
                    inter=rng.random() < 0.5, dtype=dtype, train=rng.random() < 0.5)
    Dk, Dv = rng.choice([64, 128]), rng.choice([64, 128])
    if op == "step":
        Hk = rng.randint(1, 12)
        Hv = Hk * rng.choice([1, 1, 2])
        T = rng.choice([1, 1, 1, 2, 5])
        return dict(op=op, B=_log_int(rng, 1, 256), T=T, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, dtype=dtype, slots=rng.random() < 0.5)
    Hk = rng.randint(1, 6)
    Hv = Hk * rng.choice([1, 1, 2])
    tokens = _log_int(rng, 16, min(32768 if op == "train" else 65536, 32768 * 12 // Hv))
    if rng.random() < 0.4:
        B, T, ragged = 1, tokens, rng.randint(1, min(tokens, 32))
    else:
        B = min(tokens, _log_int(rng, 1, 32))
        T, ragged = max(1, tokens // B), 0
    return dict(op=op, B=B, T=T, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, dtype=dtype, ragged=ragged,
                init=op == "prefill" and rng.random() < 0.5)


# ------------------------------------------------------------------- inputs

def _lengths(n, total, seed):
    """n uneven lengths that sum to total; one of them 0 and one of them 1 where there is room."""
    if n == 1:
        return [total]
    gen = torch.Generator().manual_seed(seed)
    w = torch.rand(n, generator=gen, dtype=torch.float64) ** 2 + 1e-3
    if n > 3:
        w[n // 2] = 0.0
    cut = torch.floor(torch.cumsum(w, 0) / w.sum() * total + 0.5).long()
    cut[-1] = total
    lens = torch.diff(cut, prepend=torch.zeros(1, dtype=torch.long))
    return [int(x) for x in lens]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = _DT[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev, dtype=torch.float32)

    st = {"case": case, "dt": dt}
    B, T = case["B"], case["T"]
    if case["op"] == "norm":
        Hq, Hk, D, R = case["Hq"], case["Hk"], case["D"], case["R"]
        # q and k as slices of one projection of the hidden state
        qk = (normal(B, T, Hq + Hk, D) * 1.5).to(dt)
        st["q"], st["k"] = qk[:, :, :Hq], qk[:, :, Hq:]
        st["wq"], st["wk"] = 1.0 + 0.2 * normal(D), 1.0 + 0.2 * normal(D)
        st["pos"] = None
        if R:
            top = T + 512
            inv = 10000.0 ** (-torch.arange(0, R // 2, device=dev, dtype=torch.float64) / (R // 2))
            ang = torch.arange(top, device=dev, dtype=torch.float64)[:, None] * inv[None, :]
            st["cos"], st["sin"] = ang.cos().float().contiguous(), ang.sin().float().contiguous()
            start = torch.randint(0, 512, (B, 1), generator=gen, device=dev)
            st["pos"] = (start + torch.arange(T, device=dev)[None, :]).to(torch.int32).contiguous()
        else:
            st["cos"] = st["sin"] = None
        st["eps"] = 1e-6
        if case["train"]:
            st["dq"], st["dk"] = normal(B, T, Hq, D).to(dt), normal(B, T, Hk, D).to(dt)
        if own:
            import fft_long_convolution_gb300 as F
            st["plan"] = F.QKNorm(D, dt, norm=case["kind"], eps=st["eps"], rotary=R, interleaved=case["inter"])
        return st

    Hk, Hv, Dk, Dv = case["Hk"], case["Hv"], case["Dk"], case["Dv"]

    def unit(*shape):
        x = normal(*shape) + 0.5 * normal(shape[0], 1, *shape[2:])  # keys of one row have something in common
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    st["q"], st["k"] = unit(B, T, Hk, Dk), unit(B, T, Hk, Dk)
    st["v"] = normal(B, T, Hv, Dv).to(dt)
    st["beta"] = torch.sigmoid(normal(B, T, Hv)).to(dt)
    rate = torch.exp(math.log(1e-3) + (math.log(0.3) - math.log(1e-3)) * uniform(Hv))  # slow and fast heads
    st["g"] = (-rate * torch.exp(0.5 * normal(B, T, Hv))).to(dt)
    st["scale"] = Dk ** -0.5
    if case["op"] == "step":
        n = B
        st["slots"] = None
        if case["slots"]:
            n = B + B // 2 + 1
            st["slots"] = torch.randperm(n, generator=gen, device=dev)[:B].to(torch.int32).contiguous()
        st["state"] = 0.1 * normal(n, Hv, Dk, Dv)
        st["next"] = st["state"].clone()  # the pool that receives the updated states
    else:
        st["offsets"], st["lens"], n = None, [T] * B, B
        if case["ragged"]:
            n = case["ragged"]
            st["lens"] = _lengths(n, T, seed)
            off = torch.zeros(n + 1, dtype=torch.long)
            off[1:] = torch.cumsum(torch.tensor(st["lens"]), 0)
            st["offsets"] = off.to(torch.int32).to(dev)
        st["state"] = 0.1 * normal(n, Hv, Dk, Dv) if case["init"] else None
        if case["op"] == "train":
            st["do"] = normal(B, T, Hv, Dv).to(dt)
    if own:
        import fft_long_convolution_gb300 as F
        st["plan"] = F.DeltaRule(Dk, Dv, dt)
    return st


# ------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if op == "norm":
        return _norm_own(state) if own else _norm_plain(state)
    if op == "step":
        return _step_own(state) if own else _step_plain(state)
    return _chunk_own(state) if own else _chunk_plain(state)


def _norm_own(s):
    p = s["plan"]
    kw = dict(wq=s["wq"], wk=s["wk"], cos=s["cos"], sin=s["sin"], positions=s["pos"])
    qo, ko = p.forward(s["q"], s["k"], **kw)
    if not s["case"]["train"]:
        return {"q": qo, "k": ko}
    dq, dk, dwq, dwk = p.backward(s["dq"], s["dk"], s["q"], s["k"], **kw)
    return {"q": qo, "k": ko, "dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def _step_own(s):
    o = s["plan"].step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], state_out=s["next"], slots=s["slots"],
                       scale=s["scale"])
    return {"o": o, "state": s["next"]}


def _chunk_own(s):
    p, args = s["plan"], (s["q"], s["k"], s["v"], s["g"], s["beta"])
    kw = dict(offsets=s["offsets"], scale=s["scale"])
    if s["case"]["op"] == "prefill":
        o, state = p.forward(*args, state=s["state"], **kw)
        return {"o": o, "state": state}
    o, _, saved = p.forward(*args, save=True, **kw)
    dq, dk, dv, dg, dbeta, _ = p.backward(s["do"], *args, saved, **kw)
    return {"o": o, "dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta}


# ------------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, inter):
    """The first 2 x (cos's width) features of x turned by the angle of (cos, sin)."""
    R = 2 * cos.shape[-1]
    if inter:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([c, d], -1).flatten(-2) if inter else torch.cat([c, d], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _norm_plain(s):
    case, dt = s["case"], s["dt"]
    rms = case["kind"] == "rms"
    cos = sin = None
    if case["R"]:
        cos, sin = s["cos"][s["pos"].long()][:, :, None], s["sin"][s["pos"].long()][:, :, None]

    def factor(x):
        m = (x * x).sum(-1, keepdim=True)
        return torch.rsqrt(m / case["D"] + s["eps"]) if rms else torch.rsqrt(m + s["eps"])

    def forward(x, w):
        x = x.float()
        z = x * factor(x) * w
        return (z if cos is None else _rotate(z, cos, sin, case["inter"])).to(dt)

    def backward(dy, x, w):
        x, dy = x.float(), dy.float()
        r = factor(x)
        dz = dy if cos is None else _rotate(dy, cos, -sin, case["inter"])
        dw = (dz * x * r).sum((0, 1, 2))
        dz = dz * w
        dx = r * dz - x * r ** 3 * (dz * x).sum(-1, keepdim=True) / (case["D"] if rms else 1)
        return dx.to(dt), dw

    out = {"q": forward(s["q"], s["wq"]), "k": forward(s["k"], s["wk"])}
    if case["train"]:
        out["dq"], dwq = backward(s["dq"], s["q"], s["wq"])
        out["dk"], dwk = backward(s["dk"], s["k"], s["wk"])
        out["dwq"], out["dwk"] = dwq, dwk
    return out


def _heads(x, Hv):
    return x.repeat_interleave(Hv // x.shape[2], dim=2) if x.shape[2] != Hv else x


def _step_plain(s):
    case = s["case"]
    Hv = case["Hv"]
    q, k, v = _heads(s["q"], Hv).float(), _heads(s["k"], Hv).float(), s["v"].float()
    g, beta = s["g"].float(), s["beta"].float()
    at = slice(None) if s["slots"] is None else s["slots"].long()
    S = s["state"][at]
    outs = []
    for t in range(case["T"]):
        S = S * g[:, t, :, None, None].exp()
        u = beta[:, t, :, None] * (v[:, t] - (k[:, t, :, :, None] * S).sum(-2))
        S = S + k[:, t, :, :, None] * u[:, :, None, :]
        outs.append(s["scale"] * (q[:, t, :, :, None] * S).sum(-2))
    s["next"][at] = S
    return {"o": torch.stack(outs, 1).to(s["dt"]), "state": s["next"]}


def _padded(s):
    """The case's sequences as rows of one length (a whole number of chunks), and where each token went."""
    dev = s["q"].device
    lens = torch.tensor(s["lens"], device=dev)
    n, top = len(s["lens"]), max(max(s["lens"]), 1)
    top = (top + _CHUNK - 1) // _CHUNK * _CHUNK
    row = torch.repeat_interleave(torch.arange(n, device=dev), lens, output_size=sum(s["lens"]))
    start = torch.cumsum(lens, 0) - lens
    col = torch.arange(sum(s["lens"]), device=dev) - start[row]

    def put(x):
        out = torch.zeros(n, top, *x.shape[2:], device=dev, dtype=torch.float32)
        out[row, col] = x.reshape(-1, *x.shape[2:]).float()
        # [sequence, head, chunk, token, ...]
        out = out.movedim(2, 1)
        return out.reshape(n, out.shape[1], top // _CHUNK, _CHUNK, *out.shape[3:]).contiguous()

    def take(x, like):
        x = x.flatten(2, 3).movedim(1, 2)
        return x[row, col].reshape(*like.shape[:2], *x.shape[2:]).to(s["dt"])

    return put, take


def _chunk_plain(s):
    case = s["case"]
    Hv, scale = case["Hv"], s["scale"]
    put, take = _padded(s)
    q, k, v = put(_heads(s["q"], Hv)), put(_heads(s["k"], Hv)), put(s["v"])
    g, beta = put(s["g"]), put(s["beta"])
    n, C = q.shape[0], _CHUNK
    nc = q.shape[2]
    idx = torch.arange(C, device=q.device)
    low, strict = idx[:, None] >= idx[None, :], idx[:, None] > idx[None, :]
    b = g.cumsum(-1)
    G, e, last = b.exp(), (b[..., -1:] - b).exp(), b[..., -1].exp()
    D = torch.where(low, b[..., :, None] - b[..., None, :], -math.inf).exp()
    A = torch.where(strict, beta[..., :, None] * D * (k @ k.transpose(-1, -2)), 0.0)
    # (I + A)^-1 by rows
    Ti = torch.eye(C, device=q.device).expand_as(A).clone()
    for i in range(1, C):
        Ti[..., i, :i] = -(A[..., i:i + 1, :i] @ Ti[..., :i, :i])[..., 0, :]
    U = Ti @ (beta[..., None] * v)
    W = Ti @ ((beta * G)[..., None] * k)
    ek = e[..., None] * k
    S = torch.zeros(n, Hv, case["Dk"], case["Dv"], device=q.device) if s["state"] is None else s["state"].clone()
    states, new = [], []
    for c in range(nc):
        states.append(S)
        new.append(U[:, :, c] - W[:, :, c] @ S)
        S = last[:, :, c, None, None] * S + ek[:, :, c].transpose(-1, -2) @ new[-1]
    S0, vn = torch.stack(states, 2), torch.stack(new, 2)
    P = scale * D * (q @ k.transpose(-1, -2))
    o = scale * G[..., None] * (q @ S0) + P @ vn
    if case["op"] == "prefill":
        return {"o": take(o, s["q"]), "state": S}

    do = put(s["do"])
    dvo = P.transpose(-1, -2) @ do
    gq = scale * (G[..., None] * q).transpose(-1, -2) @ do
    dS = torch.zeros_like(S)
    dstates, dnew = [], []
    for c in range(nc - 1, -1, -1):
        dstates.append(dS)
        dnew.append(dvo[:, :, c] + ek[:, :, c] @ dS)
        dS = last[:, :, c, None, None] * dS + gq[:, :, c] - W[:, :, c].transpose(-1, -2) @ dnew[-1]
    dSn, dvn = torch.stack(dstates[::-1], 2), torch.stack(dnew[::-1], 2)
    dR = Ti.transpose(-1, -2) @ dvn
    X = torch.where(low, scale * D * (do @ vn.transpose(-1, -2)), 0.0)
    Hm = torch.where(strict, -D * (dR @ vn.transpose(-1, -2)), 0.0)
    dq = scale * G[..., None] * (do @ S0.transpose(-1, -2)) + X @ k
    Y = -G[..., None] * (dR @ S0.transpose(-1, -2)) + Hm @ k
    dke = e[..., None] * (vn @ dSn.transpose(-1, -2))
    up = beta[..., None] * Y
    down = X.transpose(-1, -2) @ q + (beta[..., :, None] * Hm).transpose(-1, -2) @ k + dke
    dk = up + down
    dbeta = (dR * v).sum(-1) + (k * Y).sum(-1)
    db = (q * dq).sum(-1) + (k * up).sum(-1) - (k * down).sum(-1)
    db[..., -1] += (k * dke).sum((-1, -2)) + last * (S0 * dSn).sum((-1, -2))
    dg = db.flip(-1).cumsum(-1).flip(-1)

    def shared(x):
        x = x.unflatten(1, (case["Hk"], Hv // case["Hk"])).sum(2)
        return take(x, s["q"])

    return {"o": take(o, s["q"]), "dq": shared(dq), "dk": shared(dk), "dv": take(beta[..., None] * dR, s["q"]),
            "dg": take(dg, s["q"]), "dbeta": take(dbeta, s["q"])}


# ------------------------------------------------------------------- the floor

def work(case):
    B, T = case["B"], case["T"]
    if case["op"] == "norm":
        n = B * T * (case["Hq"] + case["Hk"]) * case["D"]
        once = 2 * 2 * n + (4 * B * T if case["R"] else 0)
        if not case["train"]:
            return {"bytes": once, "flops": 8 * n}
        return {"bytes": once + 3 * 2 * n, "flops": 24 * n}
    Hk, Hv, Dk, Dv = case["Hk"], case["Hv"], case["Dk"], case["Dv"]
    qk, vo = 2 * B * T * Hk * Dk * 2, 2 * B * T * Hv * Dv * 2
    gates = 2 * 2 * B * T * Hv
    flops = 6 * B * T * Hv * Dk * Dv
    if case["op"] == "step":
        return {"bytes": qk + vo + gates + 2 * 4 * B * Hv * Dk * Dv, "flops": flops}
    rows = case["ragged"] or B
    states = 4 * rows * Hv * Dk * Dv * (2 if case["init"] else 1)
    if case["op"] == "prefill":
        return {"bytes": qk + vo + gates + states, "flops": flops}
    # o written, then do read and the five gradients written
    return {"bytes": 2 * qk + 2 * vo + 2 * gates, "flops": 3 * flops}


# ------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _norm_exact(s)
    return _rule_exact(s)


def _norm_exact(s):
    case = s["case"]
    D, R = case["D"], case["R"]
    # the rotation as one matrix for each token, applied to normed rows
    first = torch.arange(0, R, 2) if case["inter"] else torch.arange(R // 2)
    second = first + 1 if case["inter"] else first + R // 2

    def turn(x, back):
        if not R:
            return x
        c, sn = s["cos"].double()[s["pos"].long()][:, :, None], s["sin"].double()[s["pos"].long()][:, :, None]
        sn = -sn if back else sn
        y = x.clone()
        y[..., first] = c * x[..., first] - sn * x[..., second]
        y[..., second] = sn * x[..., first] + c * x[..., second]
        return y

    out = {}
    for name in ("q", "k"):
        x, w = s[name].double(), s["w" + name].double()
        size = x.pow(2).mean(-1, keepdim=True) if case["kind"] == "rms" else x.pow(2).sum(-1, keepdim=True)
        norm = (size + s["eps"]).sqrt()
        out[name] = turn(x / norm * w, False)
        if case["train"]:
            dz = turn(s["d" + name].double(), True)
            hat = x / norm
            out["dw" + name] = (dz * hat).sum((0, 1, 2))
            along = (dz * w * hat).mean(-1, keepdim=True) if case["kind"] == "rms" else (dz * w * hat).sum(-1, keepdim=True)
            out["d" + name] = (dz * w - hat * along) / norm
    order = ["q", "k"] + (["dq", "dk", "dwq", "dwk"] if case["train"] else [])
    return {n: out[n] for n in order}


def _rule_exact(s):
    """Token by token, all sequences of the case side by side."""
    case = s["case"]
    Hk, Hv, Dk, Dv = case["Hk"], case["Hv"], case["Dk"], case["Dv"]
    train, step = case["op"] == "train", case["op"] == "step"
    B = case["B"]
    lens = [case["T"]] * B if step else s["lens"]
    n, top = len(lens), max(lens + [1])
    size = n * Hv * Dk * Dv * 8
    if top * (60e-6 + 10 * size / 5e12) * (6 if train else 1) > 15 or (train and size * top > 60e9):
        return None
    dev = s["q"].device
    flat = {m: s[m].double().reshape(-1, *s[m].shape[2:]) for m in ("q", "k", "v", "g", "beta") + (("do",) if train else ())}
    start = [sum(lens[:i]) for i in range(n)]
    live_at = torch.tensor(lens, device=dev)
    begin = torch.tensor(start, device=dev)
    total = flat["v"].shape[0]
    group = Hv // Hk
    head = torch.arange(Hv, device=dev) // group
    if step:
        at = torch.arange(n, device=dev) if s["slots"] is None else s["slots"].long()
        pool = s["state"].double()
        S = pool[at]
    else:
        S = torch.zeros(n, Hv, Dk, Dv, device=dev, dtype=torch.float64) if s["state"] is None else s["state"].double()
    o = torch.zeros(total, Hv, Dv, device=dev, dtype=torch.float64)
    kept = []
    for t in range(top):
        live = (live_at > t)
        tok = torch.where(live, begin + t, 0).clamp(max=max(total - 1, 0))
        on = live[:, None, None, None]
        if train:
            kept.append(S)
        kt, qt = flat["k"][tok][:, head], flat["q"][tok][:, head]
        Sd = S * flat["g"][tok].exp()[..., None, None]
        u = flat["beta"][tok][..., None] * (flat["v"][tok] - torch.einsum("nhd,nhde->nhe", kt, Sd))
        S = torch.where(on, Sd + torch.einsum("nhd,nhe->nhde", kt, u), S)
        ot = s["scale"] * torch.einsum("nhd,nhde->nhe", qt, S)
        o.index_add_(0, tok, torch.where(live[:, None, None], ot, 0.0))
    shape = s["v"].shape
    if step:
        pool[at] = S
        return {"o": o.reshape(shape), "state": pool}
    if not train:
        return {"o": o.reshape(shape), "state": S}
    grads = {m: torch.zeros_like(flat[m]) for m in ("q", "k", "v", "g", "beta")}
    dS = torch.zeros_like(S)
    zero = torch.zeros((), device=dev, dtype=torch.float64)
    for t in range(top - 1, -1, -1):
        live = (live_at > t)
        tok = torch.where(live, begin + t, 0).clamp(max=max(total - 1, 0))
        l3, l2 = live[:, None, None], live[:, None]
        kt, qt, dot = flat["k"][tok][:, head], flat["q"][tok][:, head], flat["do"][tok]
        a, bt, vt = flat["g"][tok].exp()[..., None, None], flat["beta"][tok][..., None], flat["v"][tok]
        Sd = kept[t] * a
        miss = vt - torch.einsum("nhd,nhde->nhe", kt, Sd)
        u = bt * miss
        St = Sd + torch.einsum("nhd,nhe->nhde", kt, u)
        d1 = dS + s["scale"] * torch.einsum("nhd,nhe->nhde", qt, dot)
        dqt = s["scale"] * torch.einsum("nhde,nhe->nhd", St, dot)
        du = torch.einsum("nhde,nhd->nhe", d1, kt)
        dkt = torch.einsum("nhde,nhe->nhd", d1, u) - torch.einsum("nhde,nhe->nhd", Sd, bt * du)
        d2 = d1 - torch.einsum("nhd,nhe->nhde", kt, bt * du)
        grads["q"].index_add_(0, tok, torch.where(l3, dqt.reshape(n, Hk, group, Dk).sum(2), zero))
        grads["k"].index_add_(0, tok, torch.where(l3, dkt.reshape(n, Hk, group, Dk).sum(2), zero))
        grads["v"].index_add_(0, tok, torch.where(l3, bt * du, zero))
        grads["beta"].index_add_(0, tok, torch.where(l2, (du * miss).sum(-1), zero))
        grads["g"].index_add_(0, tok, torch.where(l2, (d2 * Sd).sum((-1, -2)), zero))
        dS = torch.where(live[:, None, None, None], d2 * a, dS)
    out = {"o": o.reshape(shape)}
    for m in ("q", "k", "v", "g", "beta"):
        out["d" + m] = grads[m].reshape(s[m].shape)
    return out
