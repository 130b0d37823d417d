"""The norm and rotation on whole batches, where a group of lanes takes several
heads of a token one after another: parts of more than three heads, parts that
hold heads of q and of k, every rotation and head size of the batch kernels.

Tolerances as for single tokens: one rounding of the output (u = 2^-8 for bf16,
2^-11 for fp16 at most), and float32 sums of the weights' gradients: 2e-5.
"""
import pytest
import torch

import fft_long_convolution_gb300 as F
from _mixers import qk_norm, rel

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# 77824 / (tokens x lanes), rounded up, is the number of parts of a token's heads
CASES = [(1, 1300, 7, 4, 256, 256), (2, 1500, 7, 4, 128, 64), (1, 5000, 4, 3, 80, 40), (1, 10007, 12, 6, 64, 32),
         (3, 1700, 2, 6, 96, 0), (1, 10001, 3, 2, 24, 6), (1, 3001, 9, 1, 128, 128), (2, 5003, 0, 5, 64, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("norm,inter", [("rms", False), ("l2", True), ("l2", False), ("rms", True)])
@pytest.mark.parametrize("B,T,Hq,Hk,D,R", CASES)
def test_forward_and_backward(B, T, Hq, Hk, D, R, norm, inter, dt):
    """Slices of one projection against the 64-bit form (on the GPU)."""
    gen = torch.Generator(device="cuda").manual_seed(D + T)

    def normal(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    qk = normal(B, T, Hq + Hk, D).to(dt)
    q, k = qk[:, :, :Hq], qk[:, :, Hq:]
    dq, dk = normal(B, T, Hq, D).to(dt), normal(B, T, Hk, D).to(dt)
    wq, wk = 1 + 0.2 * normal(D), 1 + 0.2 * normal(D)
    pos = torch.randint(0, 40, (B, T), generator=gen, device="cuda").to(torch.int32)
    ang = torch.arange(40, device="cuda")[:, None] * 100.0 ** (-torch.arange(R // 2, device="cuda") / max(R // 2, 1))
    cos, sin = ang.cos().contiguous(), ang.sin().contiguous()
    plan = F.QKNorm(D, dt, norm=norm, rotary=R, interleaved=inter)
    kw = dict(wq=wq, wk=wk, cos=cos, sin=sin, positions=pos)
    qo, ko = plan.forward(q, k, **kw)
    got = plan.backward(dq, dk, q, k, **kw)
    for x, w, d, y, gx, gw in ((q, wq, dq, qo, got[0], got[2]), (k, wk, dk, ko, got[1], got[3])):
        x, w = x.double().requires_grad_(), w.double().requires_grad_()
        ref = qk_norm(x, w, norm, 1e-6, cos, sin, pos, inter)
        assert rel(y, ref.detach().cpu()) < U[dt]
        if x.numel() == 0:
            assert not bool(gw.any())
            continue
        rx, rw = torch.autograd.grad((ref * d.double()).sum(), [x, w])
        assert rel(gx, rx.cpu()) < U[dt] and rel(gw, rw.cpu()) < 2e-5
