"""How the linear attention plans its calls: scratch sizes of rows of any shape, on the
host, and the calls that such plans lead to."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import fft_long_convolution_gb300 as F
from _attention import attention_chunks, attention_grads, attention_inputs, linear_attention, rel, states

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
NAMES = ("dq", "dk", "dv", "dstate")


class PlanOnHost(ctypes.Structure):
    """What a plan holds, for the calls that need no device."""
    _fields_ = [("Dk", ctypes.c_int), ("Dv", ctypes.c_int), ("dtype", ctypes.c_int), ("device", ctypes.c_int),
                ("num_sms", ctypes.c_int), ("dev_err", ctypes.c_void_p)]


def scratch_bytes(B, T, Hk, Hv, nseq, backward, Dk=64, Dv=64, dtype=1):
    plan = PlanOnHost(Dk, Dv, dtype, 0, 152, None)
    return int(F.lib().fftconv_linattn_scratch_bytes(ctypes.addressof(plan), B, T, Hk, Hv, nseq, backward))


def sweep_of_short_rows():
    """Packed rows of few tokens (at most one for each sequence): nothing to cut, no scratch."""
    for nseq in range(1, 70):
        for T in {0, 1, nseq - 1, nseq}:
            for H in (1, 2, 7, 12, 16, 28, 29, 32, 48, 64, 85, 86, 96, 128, 300, 1000):
                for dtype in (0, 1):
                    for backward in (0, 1):
                        n = scratch_bytes(1, T, H, H, nseq, backward, dtype=dtype)
                        assert n == 0 or T > 64, (nseq, T, H, dtype, backward, n)


def test_rows_of_fewer_tokens_than_sequences():
    """In a process of its own: a division by zero ends it."""
    r = subprocess.run([sys.executable, __file__], capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": os.pathsep.join(p for p in sys.path if p)})
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("nseq", [5, 6, 7, 8, 9, 16, 31, 32, 33, 34, 64, 100, 200])
def test_long_prompts_of_any_queue_are_cut(nseq, dtype):
    """One prompt of 60000 tokens beside any number of short ones: pieces of it have states
    in scratch, in both directions."""
    for Dk, Dv in ((64, 64), (128, 64), (128, 128)):
        for Hv in (12, 24):
            for backward in (0, 1):
                assert scratch_bytes(1, 60000 + 178 * (nseq - 1), Hv, Hv, nseq, backward, Dk, Dv, dtype) > 0, (Dk, Dv, Hv, backward)


@pytest.mark.parametrize("nseq", [33, 200, 1000, 10000])
def test_scratch_is_for_the_long_prompts(nseq):
    """Pieces' states, not states of every sequence."""
    state = 12 * 128 * 128 * 4
    for backward in (0, 1):
        assert 0 < scratch_bytes(1, 60000 + 178 * (nseq - 1), 12, 12, nseq, backward, 128, 128) < 2 * 24 * state


def offsets_of(lens):
    off = torch.zeros(len(lens) + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(torch.tensor(lens), 0)
    return off


@pytest.mark.gpu
@pytest.mark.parametrize("dt", U)
@pytest.mark.parametrize("lens", [[0] * 32, [1] * 20 + [0] * 11 + [0], [0] * 15 + [20] + [0] * 16, [2, 0, 3] + [0] * 9])
def test_queues_of_mostly_empty_prompts(lens, dt):
    """Fewer tokens than sequences over many heads.  Tolerances: o and the gradients have one
    rounding at the end and one operand rounded in each term, u together; states are sums of
    one chunk, 12 2^-23 and the parts' 2^-22."""
    Hk, Hv, Dk, Dv, n, T = 48, 96, 64, 64, len(lens), sum(lens)
    ins = attention_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=n)
    do = attention_inputs(1, T, Hk, Hv, Dk, Dv, dt, seed=n + 1)[2]
    s0, ds = states(n, Hv, Dk, Dv), states(n, Hv, Dk, Dv, seed=2)
    off = offsets_of(lens).cuda()
    plan = F.LinearAttention(Dk, Dv, dt)
    dins = [x.cuda() for x in ins]
    o, s = plan.forward(*dins, state=s0.cuda(), offsets=off)
    got = plan.backward(do.cuda(), *dins, state=s0.cuda(), dstate=ds.cuda(), offsets=off)
    assert o.shape == (1, T, Hv, Dv) and s.shape == s0.shape
    at = 0
    for i, L in enumerate(lens):
        if L == 0:
            assert torch.equal(s[i].cpu(), s0[i]) and torch.equal(got[3][i].cpu(), ds[i]), i
            continue
        part = [x[:, at:at + L] for x in ins[:3]] + [ins[3]]
        ref, sref = linear_attention(*part, state=s0[i:i + 1], scale=Dk ** -0.5)
        assert rel(o[:, at:at + L], ref) < U[dt] and rel(s[i:i + 1], sref) < 4e-6, i
        r = attention_grads(*part, do[:, at:at + L], s0[i:i + 1], ds[i:i + 1], Dk ** -0.5)
        for name, x, y in zip(NAMES[:3], got, r):
            assert rel(x[:, at:at + L], y) < U[dt], (name, i)
        assert rel(got[3][i:i + 1], r[3]) < 4e-6, i
        at += L
    assert plan.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", U)
@pytest.mark.parametrize("lens,before,behind", [([70, 0, 5, 130], 9, 11), ([64], 0, 0), ([3, 1], 0, 100), ([], 20, 0), ([0], 5, 5)])
def test_parts_of_shared_heads_in_gaps(lens, before, behind, dt):
    """Parts of dq and dk for each value head are formed and read for the sequences' tokens
    alone: scratch of NaN leaves no trace, and stays NaN for the others."""
    Hk, Hv, D, n, T = 2, 6, 64, len(lens), before + sum(lens) + behind
    q, k, v, decay = (x.cuda() for x in attention_inputs(1, T, Hk, Hv, D, D, dt, seed=n))
    do = attention_inputs(1, T, Hk, Hv, D, D, dt, seed=n + 1)[2].cuda()
    off = (offsets_of(lens) + before).cuda()
    plan = F.LinearAttention(D, D, dt)
    want = plan.backward(do, q, k, v, decay, offsets=off)
    L, a = F.lib(), plan._args(q, k, v, decay, off, None)
    need = L.fftconv_linattn_scratch_bytes(plan._h, 1, T, Hk, Hv, n, 1)
    assert need == 2 * T * Hv * D * 4  # the parts, and nothing else
    scratch = torch.full((need // 4,), float("nan"), device="cuda")
    got = [torch.full_like(x, 3.0) for x in (q, k, v)]
    views = [F.View(*F._strides(x, "x", dt, x.shape)) for x in (do, *got)]
    status = L.fftconv_linattn_backward(plan._h, ctypes.byref(a), None, views[0], None, *views[1:], None, scratch.data_ptr(),
                                        need, torch.cuda.current_stream().cuda_stream)
    assert status == 0 and plan.device_status() == 0
    for x, y in zip(got, want):
        assert torch.equal(x, y) and not bool(x[:, :before].any()) and not bool(x[:, T - behind:].any())
    assert int(scratch.isnan().sum()) == 2 * (before + behind) * Hv * D


def queue_against_definition(lens, Hk, Hv, D, dt, state_tol):
    """A packed row's outputs, states and gradients against the 64-bit definition."""
    n, T = len(lens), sum(lens)
    ins = [x.cuda() for x in attention_inputs(1, T, Hk, Hv, D, D, dt, seed=n)]
    do = attention_inputs(1, T, Hk, Hv, D, D, dt, seed=n + 1)[2].cuda()
    s0, ds = states(n, Hv, D, D).cuda(), states(n, Hv, D, D, seed=3).cuda()
    off = offsets_of(lens).cuda()
    plan = F.LinearAttention(D, D, dt)
    o, s = plan.forward(*ins, state=s0, offsets=off)
    got = plan.backward(do, *ins, state=s0, dstate=ds, offsets=off)
    for i, L in enumerate(lens):
        if not L:
            assert torch.equal(s[i], s0[i]) and torch.equal(got[3][i], ds[i])
            continue
        at = slice(int(off[i]), int(off[i]) + L)
        xs = [x.double().requires_grad_() for x in (*[y[:, at] for y in ins[:3]], s0[i:i + 1])]
        ro, rs = attention_chunks(*xs[:3], ins[3], xs[3], D ** -0.5, C=200)
        assert rel(o[:, at], ro.detach()) < U[dt] and rel(s[i:i + 1], rs.detach()) < state_tol, i
        ref = torch.autograd.grad((ro * do[:, at].double()).sum() + (rs * ds[i:i + 1].double()).sum(), xs)
        for name, x, y in zip(NAMES[:3], got, ref):
            assert rel(x[:, at], y) < U[dt], (name, i)
        assert rel(got[3][i:i + 1], ref[3]) < state_tol, i
    assert plan.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", U)
@pytest.mark.parametrize("lens,Hk,Hv", [([190] * 25 + [56226] + [190] * 24, 1, 1), ([40000] + [0] * 3 + [64] * 12 + [24001] + [130] * 9, 1, 2),
                                        ([1000, 25537] + [1000] * 6, 6, 6)])
def test_rows_cut_by_their_mean_length_with_a_long_prompt(lens, Hk, Hv, dt):
    """One prompt of a queue has most of the segments, dozens of them.  States: (12 + up to
    880 chunks) 2^-23."""
    queue_against_definition(lens, Hk, Hv, 64, dt, 1.1e-4)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,B,Hv,D", [(None, 2, 2, 64), (None, 1, 6, 128), ([64] * 5 + [9000, 0, 6000], 1, 1, 128), ([6400], 1, 2, 64),
                                         ([178] * 3 + [60000] + [100, 0, 178, 64], 1, 12, 64), ([128] * 40 + [64000], 1, 12, 128),
                                         ([25600] + [64] * 40, 1, 12, 128)])
def test_scratch_is_not_left(lens, B, Hv, D):
    """Rows and queues that are cut: nothing before and behind the scratch is written."""
    dt = torch.bfloat16
    T, n, off = (sum(lens), len(lens), offsets_of(lens).cuda()) if lens else (6401, B, None)
    q, k, v, decay = (x.cuda() for x in attention_inputs(B, T, Hv, Hv, D, D, dt, seed=n))
    plan = F.LinearAttention(D, D, dt)
    want = [*plan.forward(q, k, v, decay, offsets=off), *plan.backward(v, q, k, v, decay, offsets=off)[:3]]
    L, a = F.lib(), plan._args(q, k, v, decay, off, None)
    got = [torch.empty_like(x) for x in want]
    vo, _, *vg = (F.View(*F._strides(x, "x", dt, x.shape)) if x.dtype == dt else None for x in got)
    vv = F.View(*F._strides(v, "v", dt, v.shape))
    stream = torch.cuda.current_stream().cuda_stream
    needs = [L.fftconv_linattn_scratch_bytes(plan._h, B, T, Hv, Hv, n, backward) for backward in (0, 1)]
    assert max(needs) > 0
    for backward, need in enumerate(needs):
        hold = torch.full((need + 2 * 65536,), 7, dtype=torch.uint8, device="cuda")
        at = hold.data_ptr() + 65536
        if backward:
            status = L.fftconv_linattn_backward(plan._h, ctypes.byref(a), None, vv, None, *vg, None, at, need, stream)
        else:
            status = L.fftconv_linattn_forward(plan._h, ctypes.byref(a), None, vo, got[1].data_ptr(), at, need, stream)
        assert status == 0
        assert bool((hold[:65536] == 7).all()) and bool((hold[65536 + need:] == 7).all())
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert plan.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", U)
@pytest.mark.parametrize("lens", [[178] * 3 + [60000] + [100, 0, 178, 64], [178] * 30 + [0, 50000] + [77] * 3 + [15000],
                                  [40] * 31 + [0] * 33 + [35000] + [8192] * 2 + [200] * 20])
def test_queues_with_long_prompts(lens, dt):
    """8, 36 and 87 prompts, the long ones cut.  States: (12 + up to 938 chunks) 2^-23."""
    queue_against_definition(lens, 6, 12, 64, dt, 1.2e-4)


@pytest.mark.gpu
@pytest.mark.parametrize("Hk,Hv,n", [(1, 1, 6), (6, 12, 40)])
def test_captured_queues_replay_on_other_offsets(Hk, Hv, n):
    """Segments are planned from the row's size; which prompts are cut is seen on the device."""
    dt, D, T = torch.bfloat16, 64, 40000
    q, k, v, decay = (x.cuda() for x in attention_inputs(1, T, Hk, Hv, D, D, dt, seed=n))
    s0 = states(n, Hv, D, D).cuda()
    plan = F.LinearAttention(D, D, dt)
    rest = T - 30000
    queues = [[T // n] * n, [0] * (n - 1) + [T], [30000] + [rest // (n - 1)] * (n - 1), [rest // (n - 1)] * (n - 1) + [30000], [0] * n]
    off = offsets_of(queues[0]).cuda()

    def work():
        o, s = plan.forward(q, k, v, decay, state=s0, offsets=off)
        return [o, s, *plan.backward(v, q, k, v, decay, state=s0, dstate=s0, offsets=off)]

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = work()
    for lens in queues:
        off.copy_(offsets_of(lens))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(kept, work()))
        for x in (kept[0], *kept[2:5]):
            assert not bool(x[:, sum(lens):].any())
    assert torch.equal(kept[1], s0) and torch.equal(kept[5], s0) and plan.device_status() == 0


if __name__ == "__main__":
    sweep_of_short_rows()
