"""What the gated delta rule promises beside its values: overlaps, calls without
value heads."""
import ctypes

import pytest
import torch

import fft_long_convolution_gb300 as F
from _mixers import delta_inputs


@pytest.mark.gpu
@pytest.mark.parametrize("over", ["dq", "dv", "dbeta", "dstate"])
def test_scratch_and_state_gradient_over_outputs_are_refused(over):
    dt, B, T, H, D = torch.bfloat16, 2, 70, 2, 64
    q, k, v, g, beta = (x.cuda() for x in delta_inputs(B, T, H, H, D, D, dt))
    plan = F.DeltaRule(D, D, dt)
    _, _, saved = plan.forward(q, k, v, g, beta, save=True)
    args = plan._args(q, k, v, g, beta, None, None)
    need = F.lib().fftconv_delta_scratch_bytes(plan._h, B, T, H, H, B, 1)
    big = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    outs = {n: torch.zeros_like(x) for n, x in zip(("dq", "dk", "dv", "dg", "dbeta"), (q, k, v, g, beta))}
    dstate = torch.zeros(B, H, D, D, device="cuda")

    def call(scratch, ds):
        views = [F.View(t.data_ptr(), *t.stride()[:3]) for t in outs.values()]
        do = F.View(v.data_ptr(), *v.stride()[:3])
        return F.lib().fftconv_delta_backward(plan._h, ctypes.byref(args), do, None, saved.data_ptr(), *views, ds, scratch, need,
                                              None)

    # the output in the middle of what is scratch (or, for a tokens' gradient, of the state's)
    at = big[1 << 12:]
    if over == "dstate":
        assert call(big.data_ptr(), at.data_ptr()) == 1
    else:
        t = outs[over]
        outs[over] = at[:t.numel() * 2].view(dt).view(t.shape)
        assert call(big.data_ptr(), dstate.data_ptr()) == 1
        scratch = torch.zeros(need, dtype=torch.uint8, device="cuda")
        assert call(scratch.data_ptr(), at[:-16].data_ptr() - 64) == 1
        torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("B,offsets", [(2, None), (1, None), (1, [3, 20])])
def test_no_value_heads(B, offsets):
    """Queries and keys that no value head uses have zero gradients."""
    dt, T, Hk, D = torch.bfloat16, 30, 2, 64
    q, k, v, g, beta = (x.cuda() for x in delta_inputs(B, T, Hk, Hk, D, D, dt))
    v, g, beta = v[:, :, :0], g[:, :, :0], beta[:, :, :0]
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda()
    plan = F.DeltaRule(D, D, dt)
    o, s, saved = plan.forward(q, k, v, g, beta, offsets=off, save=True)
    assert o.shape == v.shape and s.shape == (B, 0, D, D)
    for _ in range(2):
        # what the allocator hands out next is not zero
        keep = [torch.full((B, T, Hk, D), 3.0, dtype=dt, device="cuda") for _ in range(4)]
        del keep
        got = plan.backward(o, q, k, v, g, beta, saved, offsets=off)
        assert got[0].shape == q.shape and not bool(got[0].any()) and not bool(got[1].any())
