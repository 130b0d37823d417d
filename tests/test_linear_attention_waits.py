"""The walks' roles hand over through barriers: every answer of a poll is voted on by its
warp, and walks whose copies are late (another stream keeps the memory busy) give the bits
of undisturbed ones."""
import os
import re

import pytest
import torch

import fft_long_convolution_gb300 as F
from _attention import attention_inputs, states

CSRC = os.path.join(os.path.dirname(os.path.abspath(F.__file__)), "csrc")


def test_polls_are_voted_on():
    """mbarrier.try_wait answers each lane by itself; .sync.aligned instructions follow."""
    with open(os.path.join(CSRC, "linattn_chunk.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert text.count("try_wait") == 1
    lines = text.split("\n")
    uses = [i for i, line in enumerate(lines) if re.search(r"(?<!bool )\bpoll\(", line)]
    assert uses
    for i in uses:  # voted on at once, or all of a line's answers on the next line
        names = re.findall(r"(\w+) = poll\(", lines[i])
        vote = f"__all_sync(0xffffffffu, {' && '.join(names)})" if names else "__all_sync(0xffffffffu, poll("
        assert vote in lines[i + 1 if names else i], lines[i]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_walks_beside_a_busy_memory(Dk, Dv, dt):
    Hk, Hv, lens = 6, 12, [700, 64, 1, 0, 2999, 130, 63, 4000]
    T, n = sum(lens), len(lens)
    ins = [x.cuda() for x in attention_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=5)]
    do = attention_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=6)[2].cuda()
    s0, ds = states(n, Hv, Dk, Dv).cuda(), states(n, Hv, Dk, Dv, seed=7).cuda()
    off = torch.zeros(n + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(torch.tensor(lens), 0)
    off = off.cuda()
    plan = F.LinearAttention(Dk, Dv, dt)

    def work():
        return [*plan.forward(*ins, state=s0, offsets=off), *plan.backward(do, *ins, state=s0, dstate=ds, offsets=off)]

    want = work()
    src = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    dst = torch.empty_like(src)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(60):
            dst.copy_(src)
    got = [work() for _ in range(6)]
    torch.cuda.synchronize()
    assert plan.device_status() == 0
    assert all(torch.equal(x, y) for g in got for x, y in zip(g, want))
