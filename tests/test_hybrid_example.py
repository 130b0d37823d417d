"""The hybrid mixer example: the operators together with a long convolution."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_hybrid_mixer():
    """The loss falls; tokens decoded one by one agree with the prompt run as a
    whole to the rounding of the outputs (both within 1.25 u of the same values,
    u = 2^-8)."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import hybrid_mixer
    finally:
        sys.path.pop(0)
    r = hybrid_mixer.run(batch=2, tokens=1024, steps=4, hidden=512, decode=5)
    assert r["shape"] == (2, 1024, 512)
    assert r["losses"][-1] < r["losses"][0]
    assert r["decode_difference"] < 2.5 * 2.0 ** -8


@pytest.mark.gpu
def test_captured_calls():
    """After a first call every call can be captured: a decoding step (norm, then
    the recurrent step) and a training step replay to the same bits."""
    import torch

    import fft_long_convolution_gb300 as F

    gen = torch.Generator(device="cuda").manual_seed(3)

    def randn(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    norm, rule = F.QKNorm(64, torch.bfloat16, norm="l2", rotary=32), F.DeltaRule(64, 128, torch.bfloat16)
    cos, sin = randn(8, 16).cos(), randn(8, 16).sin()
    state = randn(3, 4, 64, 128)
    out = torch.empty_like(state)

    def inputs(T):
        return (randn(3, T, 2, 64).bfloat16(), randn(3, T, 2, 64).bfloat16(), randn(3, T, 4, 128).bfloat16(),
                (-randn(3, T, 4).abs()).bfloat16(), torch.sigmoid(randn(3, T, 4)).bfloat16())

    one, many = inputs(1), inputs(150)

    def decode():
        q, k, v, g, beta = one
        q, k = norm.forward(q, k, cos=cos, sin=sin)
        return rule.step(q, k, v, g, beta, state, state_out=out)

    def train():
        q, k, v, g, beta = many
        k = torch.nn.functional.normalize(k.float(), dim=-1).bfloat16()
        o, _, saved = rule.forward(q, k, v, g, beta, state=state, save=True)
        return o, *rule.backward(v, q, k, v, g, beta, saved)

    for call in (lambda: (decode(), out.clone()), train):
        want = call()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            got = call()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert rule.device_status() == 0
